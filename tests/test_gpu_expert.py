"""The expert layer's operators on the GPU against their 64-bit definitions.

Bounds come from the formats (see expert_reference); outputs are framed by
guard elements that must stay as they were."""
import math

import pytest

torch = pytest.importorskip("torch")

import expert_reference as ref  # noqa: E402
import ffn_reference  # noqa: E402
import layout_aware_collectives_gb300 as tide  # noqa: E402
from test_gpu_compute import Guarded, close, gen, strided  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def compute():
    with tide.Compute() as c:
        yield c


def randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def out_i32(*shape):
    n = 1
    for s in shape[1:]:
        n *= s
    return Guarded(shape[0], n, dtype=torch.int32)


def same(got, want):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    return torch.nan_to_num(got), torch.nan_to_num(want)


# ------------------------------------------------------------------- routing

ROUTERS = [
    dict(experts=1, topk=1), dict(experts=8, topk=2), dict(experts=60, topk=4, score="sigmoid"),
    dict(experts=128, topk=8), dict(experts=128, topk=8, renormalize=False, scale=0.5),
    dict(experts=160, topk=6, groups=8, top_groups=3), dict(experts=256, topk=8, score="sigmoid", groups=8, top_groups=4, group_best=2, scale=2.5),
    dict(experts=100, topk=16, groups=4, top_groups=2, group_best=2, renormalize=False), dict(experts=33, topk=16),
    dict(experts=32, topk=4, groups=32, top_groups=5, group_best=2), dict(experts=1024, topk=16, score="sigmoid", renormalize=False),
    dict(experts=512, topk=10, groups=2, top_groups=1, group_best=2), dict(experts=14, topk=3, groups=7, top_groups=2),
]


def check_route(compute, router, logits, bias, kind, pad=0):
    t, e = logits.shape
    r = tide.Router(**router)
    ids, w = out_i32(t, r.topk), Guarded(t, r.topk, dtype=torch.float32)
    compute.route(r, t, strided(logits, e + pad) if pad else logits, ids, w, bias=bias, logits_type=kind, ld_logits=e + pad)
    opts = {k: v for k, v in router.items() if k not in ("experts", "topk")}
    want_ids, want_w = ref.route(logits, r.topk, bias=bias, **opts)
    assert torch.equal(ids.view, want_ids.int())
    got, want = same(w.view, want_w)
    close(got, want, ref.route_bound(logits, want_ids, want, router.get("score", "softmax")))
    assert ids.intact() and w.intact()


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(compute, router, kind, biased):
    for tokens, pad in ((1, 0), (3, 1), (37, 0), (1021, 4)):
        g = gen(tokens + router["experts"])
        logits = randn(g, tokens, router["experts"], scale=1.5, dtype=TYPES[kind])
        bias = randn(g, router["experts"], scale=0.05) if biased else None
        check_route(compute, router, logits, bias, kind, pad)


@pytest.mark.parametrize("router", ROUTERS)
def test_route_ties_and_masks(compute, router):
    """Few different values, masked experts, rows with none left, saturated scores."""
    g = gen(11)
    e = router["experts"]
    logits = torch.randint(-2, 3, (200, e), generator=g, device="cuda").float()
    logits[torch.rand(200, e, generator=g, device="cuda") < 0.3] = -math.inf
    logits[7] = -math.inf
    logits[8] = 0.0
    logits[9] = -0.0
    logits[9, ::2] = 0.0
    logits[10] = 30 + torch.arange(e, device="cuda") % 3
    logits[11] = -200 - torch.arange(e, device="cuda") % 5
    logits[12] = 1e30
    logits[13] = -1e30
    check_route(compute, router, logits, None, "fp32")
    bias = torch.randint(-1, 2, (e,), generator=g, device="cuda").float() / 8
    check_route(compute, router, logits, bias, "fp32")
    check_route(compute, router, logits, torch.zeros(e, device="cuda"), "fp32")
    bias[::3] = -math.inf
    check_route(compute, router, logits, bias, "fp32")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("levels,e", [(8, 64), (1, 64), (3, 32), (2, 256), (1, 20)])
def test_route_borders_that_32_bits_do_not_tell(compute, score, levels, e):
    """Score plus bias of neighbours a few 2^-26 apart, in 64 bits and no further:
    of a few, and of more than a warp has lanes."""
    g = gen(12)
    t = 300
    logits = randn(g, 1, e).repeat(t, 1)
    s = ref.scores(logits, score)
    # each expert's bias brings it to one of the levels, as near as fp32 has it
    level = torch.arange(e, device="cuda") % levels / 16 + 1
    bias = (level - s[0]).float()
    logits = (logits.double() + torch.randn(t, e, generator=g, device="cuda", dtype=torch.float64) * 1e-7).float()
    check_route(compute, dict(experts=e, topk=16, score=score, renormalize=False), logits, bias, "fp32")
    check_route(compute, dict(experts=e, topk=6, score=score, groups=4, top_groups=2, group_best=2), logits, bias, "fp32")
    check_route(compute, dict(experts=e, topk=3, score=score, groups=4, top_groups=3), logits, bias, "fp32")


@pytest.mark.parametrize("top", [40.0, 1.0, 0.0, -1.0, -30.0, -59.0, -61.0, -85.0, -200.0])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_route_shares_of_far_sigmoids(compute, top, kind):
    """Sigmoids' shares down to where fp32 ends, though the sigmoids themselves do
    not reach as far: forward and back."""
    g = gen(16)
    t, e, k = 100, 12, 6
    logits = top - 70 * torch.rand(t, e, generator=g, device="cuda")
    logits[:, 3] = top
    logits[1, 5:] = -math.inf
    logits[2, 4:], logits[2, :3] = -math.inf, -math.inf
    logits[3] = -math.inf
    logits = logits.to(TYPES[kind])
    router = dict(experts=e, topk=k, score="sigmoid", scale=2.5)
    check_route(compute, router, logits, None, kind)
    check_route(compute, router, logits, torch.zeros(e, device="cuda"), kind)
    ids = ref.route(logits, k, score="sigmoid")[0].int().contiguous()
    dw, out = randn(g, t, k), Guarded(t, e, dtype=TYPES[kind])
    compute.route_backward(tide.Router(**router), t, logits, ids, dw, out, logits_type=kind)
    want, bound = ref.route_backward(logits, ids, dw, "sigmoid", True, 2.5)
    close(out.view, want, bound + (ref.U_BF16 * (want.abs() + bound) if kind == "bf16" else 0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups", [(256, 8), (100, 4), (64, 32)])
@pytest.mark.parametrize("size", [4.0, 64.0, 1000.0, 1e6, 2e38])
def test_route_groups_whose_terms_cancel(compute, score, experts, groups, size):
    """Groups of two large biases of opposite signs, whose sum is small and whose
    roundings are not, a few 1e-5 and less from one another."""
    g = gen(14)
    t, each = 400, experts // groups
    noise = torch.exp(3 * torch.randn(t, 1, generator=g, device="cuda", dtype=torch.float64)) * 1e-6
    logits = (0.5 + noise * torch.randn(t, experts, generator=g, device="cuda", dtype=torch.float64)).float()
    bias = torch.full((groups, each), -1.5 * size, device="cuda")
    bias[:, each // 2], bias[:, 0] = size, -size
    if size > 1e38:  # two terms of one sign, whose sum leaves fp32
        bias[:, 0] = size
    kept = max(1, groups // 2)
    check_route(compute, dict(experts=experts, topk=2, score=score, groups=groups, top_groups=kept, group_best=2), logits, bias.view(-1), "fp32")


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("biased", [False, True])
def test_route_not_finite(compute, router, biased):
    """NaN and infinite logits: ids are valid and distinct, NaN where the formula has it."""
    g = gen(13)
    e, t = router["experts"], 60
    r = tide.Router(**router)
    logits = randn(g, t, e)
    flat = logits.view(-1)
    for v in (math.nan, math.inf, -math.inf):
        flat[torch.randint(0, flat.numel(), (t,), generator=g, device="cuda")] = v
    logits[0], logits[1] = math.nan, math.inf
    bias = randn(g, e, scale=0.1) if biased else None
    if biased:
        bias[e // 2] = math.nan
        bias[0] = math.inf
    ids, w = out_i32(t, r.topk), Guarded(t, r.topk, dtype=torch.float32)
    compute.route(r, t, logits, ids, w, bias=bias)
    got = ids.view.long()
    assert int(got.min()) >= 0 and int(got.max()) < e
    ordered = torch.sort(got, dim=1).values
    assert not bool((ordered[:, 1:] == ordered[:, :-1]).any())
    if router.get("score") != "sigmoid":
        bad = torch.isnan(logits).any(1) | (logits == math.inf).any(1)
        assert torch.equal(torch.isnan(w.view).all(1), bad) and torch.equal(torch.isnan(w.view).any(1), bad)
    assert ids.intact() and w.intact()


@pytest.mark.parametrize("router", [r for r in ROUTERS if r["experts"] != 1])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_route_backward(compute, router, kind):
    e, k = router["experts"], router["topk"]
    r = tide.Router(**router)
    score, renorm, scale = router.get("score", "softmax"), router.get("renormalize", True), router.get("scale", 1.0)
    for tokens, pad in ((1, 0), (3, 1), (37, 0), (259, 4)):
        g = gen(tokens + e + 1)
        logits = randn(g, tokens, e, scale=2.0, dtype=TYPES[kind])
        ids = torch.topk(logits.float(), k, dim=1).indices.int()
        if tokens > 30:
            ids[3, 0], ids[4, -1] = -1, e  # no expert
            ids[5, 0] = ids[5, -1]  # twice
            logits[6] = -math.inf
            logits[7, : e // 2] = -math.inf
            logits[8], logits[9] = -300.0, 100.0
        dw = randn(g, tokens, k)
        out = Guarded(tokens, e, e + pad, dtype=TYPES[kind])
        compute.route_backward(r, tokens, strided(logits, e + pad) if pad else logits, ids, dw, out, logits_type=kind, ld_logits=e + pad,
                               ld_dlogits=e + pad)
        want, bound = ref.route_backward(logits, ids, dw, score, renorm, scale)
        if kind == "bf16":
            bound = bound + ref.U_BF16 * (want.abs() + bound)
        close(out.view, want, bound)
        assert out.intact()


# ------------------------------------------------------------- expert order

@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 128), (37, 8, 128), (255, 8, 3), (257, 8, 60), (2048, 1, 1024), (8191, 8, 128),
                                                 (70001, 2, 7), (100000, 10, 300), (3, 1000, 50)])
@pytest.mark.parametrize("missing", [False, True])
def test_slots(compute, tokens, topk, experts, missing):
    g = gen(tokens)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda", dtype=torch.int32)
    if missing:
        ids[torch.rand(tokens, topk, generator=g, device="cuda") < 0.2] = -1
        ids[-1, -1] = experts
        ids[0, 0] = -2 ** 31
    slots, offsets = out_i32(tokens, topk), out_i32(1, experts + 1)
    ws = torch.empty(tide.expert_slots_workspace_bytes(tokens, topk, experts), dtype=torch.uint8, device="cuda")
    compute.expert_slots(tokens, topk, experts, ids, slots, offsets, ws)
    want_slots, want_offsets = ref.slots(ids, experts)
    assert torch.equal(slots.view.cpu(), want_slots) and torch.equal(offsets.view.cpu().view(-1), want_offsets)
    assert slots.intact() and offsets.intact()


def test_slots_of_no_tokens(compute):
    offsets = out_i32(1, 9)
    compute.expert_slots(0, 2, 8, 0, 0, offsets, 0, workspace_bytes=0)
    assert not bool(offsets.view.any()) and offsets.intact()


# ---------------------------------------------------------------- the rows

ROWS = [(1, 8, 1), (1, 2048, 8), (37, 2048, 8), (5, 1, 3), (300, 250, 2), (64, 1024, 10), (33, 4096, 17), (129, 40, 9), (7, 8200, 4), (20, 777, 8)]


def some_slots(g, tokens, topk, rows, missing):
    at = torch.randperm(rows, generator=g, device="cuda")[: tokens * topk].view(tokens, topk).int()
    if missing:
        at[torch.rand(tokens, topk, generator=g, device="cuda") < 0.2] = -1
        at[0, -1] = rows
    return at.contiguous()


@pytest.mark.parametrize("tokens,hidden,topk", ROWS)
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("missing", [False, True])
def test_gather(compute, tokens, hidden, topk, pad, missing):
    g = gen(tokens + hidden)
    n = tokens * topk + 5
    x = randn(g, tokens, hidden, dtype=torch.bfloat16)
    slots = some_slots(g, tokens, topk, n, missing)
    rows = Guarded(n, hidden, hidden + pad)
    before = rows.view.clone()
    compute.expert_gather(tokens, hidden, topk, strided(x, hidden + pad) if pad else x, slots, rows, n, ld_x=hidden + pad, ld_rows=hidden + pad)
    want = before
    inside = (slots >= 0) & (slots < n)
    want[slots[inside].long()] = x.repeat_interleave(topk, 0)[inside.view(-1)]
    assert torch.equal(rows.view.view(torch.int16), want.view(torch.int16))
    assert rows.intact()


@pytest.mark.parametrize("tokens,hidden,topk", ROWS)
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("weighted,missing", [(True, False), (True, True), (False, True)])
def test_combine(compute, tokens, hidden, topk, pad, weighted, missing):
    g = gen(tokens + hidden + 1)
    n = tokens * topk + 5
    rows = randn(g, n, hidden, dtype=torch.bfloat16)
    slots = some_slots(g, tokens, topk, n, missing)
    if missing:
        rows[~torch.isin(torch.arange(n, device="cuda"), slots)] = math.nan  # rows of nobody's are not read
    w = randn(g, tokens, topk) if weighted else None
    y = Guarded(tokens, hidden, hidden + pad)
    compute.expert_combine(tokens, hidden, topk, strided(rows, hidden + pad) if pad else rows, n, slots, w, y, ld_rows=hidden + pad,
                           ld_y=hidden + pad)
    close(y.view, *ref.combine(torch.nan_to_num(rows), slots, w))
    assert y.intact()


@pytest.mark.parametrize("tokens,hidden,topk", ROWS)
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("weighted,missing", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("outputs", ["both", "rows", "weights"])
def test_combine_backward(compute, tokens, hidden, topk, pad, weighted, missing, outputs):
    g = gen(tokens + hidden + 2)
    n = tokens * topk + 5
    rows, dy = randn(g, n, hidden, dtype=torch.bfloat16), randn(g, tokens, hidden, dtype=torch.bfloat16)
    slots = some_slots(g, tokens, topk, n, missing)
    w = randn(g, tokens, topk) if weighted else None
    drows, dw = Guarded(n, hidden, hidden + pad), Guarded(tokens, topk, dtype=torch.float32)
    before = drows.view.clone()
    compute.expert_combine_backward(tokens, hidden, topk, strided(dy, hidden + pad) if pad else dy,
                                    None if outputs == "rows" else strided(rows, hidden + pad) if pad else rows, n, slots, w,
                                    None if outputs == "weights" else drows, None if outputs == "rows" else dw, ld_dy=hidden + pad,
                                    ld_rows=hidden + pad, ld_drows=hidden + pad)
    each, each_bound, want_dw, dw_bound = ref.combine_backward(dy, rows, slots, w)
    inside = (slots >= 0) & (slots < n)
    if outputs != "weights":
        close(drows.view[slots[inside].long()], each[inside], each_bound[inside])
        rest = ~torch.isin(torch.arange(n, device="cuda"), slots)
        assert torch.equal(drows.view[rest].view(torch.int16), before[rest].view(torch.int16))
    if outputs != "rows":
        close(dw.view, want_dw, dw_bound)
    assert drows.intact() and dw.intact()


def among_nan(x, ld):
    """x's rows `ld` apart, NaN between them and nothing behind the last."""
    held = torch.full(((x.shape[0] - 1) * ld + x.shape[1],), math.nan, dtype=x.dtype, device="cuda")
    view = held.as_strided(x.shape, (ld, 1))
    view.copy_(x)
    return view


@pytest.mark.parametrize("hidden", [1, 7, 9, 511, 512, 513, 517, 520, 1035])
@pytest.mark.parametrize("topk", [1, 3, 9])
@pytest.mark.parametrize("pads", [(0, 1), (1, 0), (3, 6), (2, 5), (7, 7)])
def test_rows_from_any_element_on(compute, hidden, topk, pads):
    """Rows of the tokens and of the experts that start on other parts of 16
    bytes, there, back and backward; what lies between rows is neither used nor written."""
    g = gen(hidden + topk)
    tokens = 19
    n = tokens * topk + 2
    ld_t, ld_r = hidden + pads[0], hidden + pads[1]
    x, rows = randn(g, tokens, hidden, dtype=torch.bfloat16), randn(g, n, hidden, dtype=torch.bfloat16)
    slots = some_slots(g, tokens, topk, n, False)
    slots[0, 0], slots[-1, -1] = n - 1, 0  # both ends, once each
    used, count = torch.unique(slots, return_counts=True)
    for twice in used[count > 1]:  # a slot that this left to two pairs goes to the first
        at = (slots == twice).nonzero()
        keep = 0 if twice == n - 1 else len(at) - 1
        for i, (a, b) in enumerate(at.tolist()):
            if i != keep:
                slots[a, b] = -1
    inside = slots >= 0
    w = randn(g, tokens, topk)
    got = Guarded(n, hidden, ld_r)
    want = got.view.clone()
    compute.expert_gather(tokens, hidden, topk, among_nan(x, ld_t), slots, got, n, ld_x=ld_t, ld_rows=ld_r)
    want[slots[inside].long()] = x.repeat_interleave(topk, 0)[inside.view(-1)]
    assert torch.equal(got.view.view(torch.int16), want.view(torch.int16)) and got.intact()
    y = Guarded(tokens, hidden, ld_t)
    compute.expert_combine(tokens, hidden, topk, among_nan(rows, ld_r), n, slots, w, y, ld_rows=ld_r, ld_y=ld_t)
    close(y.view, *ref.combine(rows, slots, w))
    assert y.intact()
    drows, dw = Guarded(n, hidden, ld_t), Guarded(tokens, topk, dtype=torch.float32)
    compute.expert_combine_backward(tokens, hidden, topk, among_nan(x, ld_t), among_nan(rows, ld_r), n, slots, w, drows, dw, ld_dy=ld_t,
                                    ld_rows=ld_r, ld_drows=ld_t)
    each, each_bound, want_dw, dw_bound = ref.combine_backward(x, rows, slots, w)
    close(drows.view[slots[inside].long()], each[inside], each_bound[inside])
    close(dw.view, want_dw, dw_bound)
    assert drows.intact() and dw.intact()


# ------------------------------------------------------- orthogonalisation

MATRICES = [(1, 1, 1), (1, 1, 7), (2, 7, 1), (3, 5, 9), (1, 64, 64), (2, 65, 130), (1, 300, 77), (1, 704, 256), (3, 250, 250), (2, 128, 1000),
            (1, 513, 1024), (1, 1021, 333), (5, 256, 257), (1, 8, 5000), (4, 384, 512),
            (1, 3457, 63), (7, 33, 2500), (16, 300, 300), (2, 64, 65), (1, 129, 4097)]


def gradients(g, count, rows, cols, kind):
    m = randn(g, count, rows, cols) + torch.bmm(randn(g, count, rows, 2), randn(g, count, 2, cols))
    return [v.contiguous() for v in (m * torch.exp(2 * randn(g, count, 1, 1)) * 1e-3).to(TYPES[kind]).unbind(0)]


def orthogonalized(compute, grads, kind="fp32", pad=0, **kw):
    rows, cols = grads[0].shape
    outs = [Guarded(rows, cols, cols + pad) for _ in grads]
    ws = torch.empty(tide.orthogonalize_workspace_bytes(len(grads), rows, cols), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # NaN wherever it is read before it is written
    src = [strided(v, cols + pad) for v in grads] if pad else grads
    compute.orthogonalize(rows, cols, src, outs, ws, src_type=kind, ld_src=cols + pad, ld_dst=cols + pad, **kw)
    assert all(o.intact() for o in outs)
    return [o.view for o in outs]


def near(got, grad, **kw):
    """The error's norm: the products' bound and the result's rounding."""
    want = ref.orthogonalize(grad, **kw)
    bound = ref.orthogonalize_bound(grad, **kw) + ref.U_BF16 * float(want.norm()) + ref.TINY
    assert bool(torch.isfinite(got).all())
    off = float((got.double() - want).norm())
    assert off <= bound, (off, bound, float(want.norm()))


@pytest.mark.parametrize("count,rows,cols", MATRICES)
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
def test_orthogonalize(compute, count, rows, cols, kind, pad):
    grads = gradients(gen(rows + cols), count, rows, cols, kind)
    for got, grad in zip(orthogonalized(compute, grads, kind, pad), grads):
        near(got, grad)


@pytest.mark.parametrize("rows,cols", [(512, 512), (384, 1024), (1024, 400), (256, 704)])
def test_orthogonalize_is_as_near_as_bf16_is(compute, rows, cols):
    """What the products leave is at most the result's own rounding, and independent of it."""
    for kind in ("fp32", "bf16"):
        grad = gradients(gen(rows), 1, rows, cols, kind)[0]
        want = ref.orthogonalize(grad)
        off = (orthogonalized(compute, [grad], kind)[0].double() - want).norm()
        assert float(off) <= math.sqrt(2) * float((want.bfloat16().double() - want).norm())


@pytest.mark.parametrize("rows,cols", [(96, 200), (200, 96), (128, 150)])
@pytest.mark.parametrize("kw", [dict(steps=0), dict(steps=1), dict(steps=2), dict(steps=10, coefficients=(1.5, -0.5, 0.0)),
                                dict(steps=8, coefficients=(1.875, -1.25, 0.375)), dict(steps=3, coefficients=(2.0, 0.0, -0.5)),
                                dict(steps=2, coefficients=(4.0, -6.0, 2.5, 3.0, -3.5, 1.25)), dict(eps=0.0), dict(eps=10.0),
                                dict(steps=4, coefficients=(0.0, 0.0, 0.0)), dict(steps=5, coefficients=(6.0, 0.0, 0.0)),
                                dict(steps=3, coefficients=(8.0, -22.0, 16.0, 2.5, -1.0, 0.1, 1.875, -1.25, 0.375))])
def test_orthogonalize_steps(compute, rows, cols, kw):
    grads = gradients(gen(3), 2, rows, cols, "fp32")
    for got, grad in zip(orthogonalized(compute, grads, **kw), grads):
        near(got, grad, **kw)


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-12, 1e12, 1e30, 3e37])
def test_orthogonalize_magnitudes(compute, scale):
    """Gradients at both ends of fp32: the norm neither vanishes nor overflows."""
    g = gen(4)
    grad = (torch.randn(70, 90, generator=g, device="cuda", dtype=torch.float64) * scale).float()
    near(orthogonalized(compute, [grad], eps=0.0)[0], grad, eps=0.0)
    near(orthogonalized(compute, [grad])[0], grad)


def spectra(g, rows, cols, kind):
    """Noise, noise over rank one, spectra of e^-4 to e^-14, columns of very different sizes."""
    m = min(rows, cols)
    one = randn(g, rows, 1) @ randn(g, 1, cols)
    out = [randn(g, rows, cols)] + [one + 10.0 ** -e * randn(g, rows, cols) for e in (1, 2, 3, 4, 5)]
    u, v = (torch.linalg.qr(torch.randn(n, m, generator=g, device="cuda", dtype=torch.float64))[0] for n in (rows, cols))
    for depth in (4, 8, 14):
        s = torch.exp(-depth * torch.arange(m, device="cuda", dtype=torch.float64) / max(1, m - 1))
        out.append((u * s) @ v.T)
    out.append(randn(g, rows, cols) * torch.exp(3 * randn(g, 1, cols)))
    return [v.to(TYPES[kind]).contiguous() for v in out]


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (2, 3), (2, 50), (50, 3), (5, 5), (8, 8), (8, 5000), (15, 100), (16, 16), (16, 64), (3000, 16),
                                       (16, 70001), (1 << 20, 4), (1, 300000)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
def test_orthogonalize_short_sides(compute, rows, cols, kind, pad):
    """Up to 16 rows or columns: 32-bit arithmetic, whatever the spectrum.  Five steps
    stretch by 485 at most what roundings of 2^-24 and sums of 16 terms leave in each."""
    grads = spectra(gen(rows + 3 * cols), rows, cols, kind)
    for got, grad in zip(orthogonalized(compute, grads, kind, pad), grads):
        want = ref.orthogonalize(grad)
        size, own = float(want.norm()), float((want.bfloat16().double() - want).norm())
        # 2^-24 * 485 * (a few roundings in each of five steps): 2^-12
        assert float((got.double() - want).norm()) <= own + 2.0 ** -12 * size


@pytest.mark.parametrize("count,rows,cols", [(300, 3, 40), (130, 70, 9), (2000, 16, 16), (1, 16, 1 << 18), (70, 8, 9000)])
def test_orthogonalize_short_sides_of_many(compute, count, rows, cols):
    """As many as several launches take, each as alone; in place too; the same bits every time."""
    grads = gradients(gen(18), count, rows, cols, "bf16")
    got = orthogonalized(compute, grads, "bf16")
    for i in sorted({0, count // 2, count - 1}):
        near(got[i], grads[i])
        assert torch.equal(orthogonalized(compute, [grads[i]], "bf16")[0], got[i])
    assert all(torch.equal(a, b) for a, b in zip(orthogonalized(compute, grads, "bf16"), got))
    ws = torch.empty(tide.orthogonalize_workspace_bytes(count, rows, cols), dtype=torch.uint8, device="cuda")
    own = [v.clone() for v in grads]
    compute.orthogonalize(rows, cols, own, own, ws)
    assert all(torch.equal(a, b) for a, b in zip(own, got))


@pytest.mark.parametrize("rows,cols", [(17, 40), (17, 17), (33, 2500), (32, 32), (64, 64), (64, 200), (200, 65), (65, 66), (128, 150), (128, 1000), (300, 256),
                                       (256, 704), (383, 1000), (384, 1024), (512, 1024), (640, 960), (1100, 700), (768, 2048),
                                       (1024, 1536), (2200, 800)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_orthogonalize_leaves_what_is_documented(compute, rows, cols, kind):
    """2^-9 of the result's norm, whatever the spectrum, a quarter more where steps
    share a pass over X.  By the 64-bit result alone."""
    m = min(rows, cols)
    limit = 2.0 ** -9 * (1.25 if m >= 384 and 2 * max(rows, cols) >= 5 * m else 1)
    grads = spectra(gen(rows + 3 * cols), rows, cols, kind)
    worst = []
    for got, grad in zip(orthogonalized(compute, grads, kind), grads):
        want = ref.orthogonalize(grad)
        size, own = float(want.norm()), float((want.bfloat16().double() - want).norm())
        # the result's rounding comes on top, independent of it where there are many elements
        most = math.hypot(own, limit * size) if want.numel() >= 1024 else own + limit * size
        worst.append(float((got.double() - want).norm()) / most)
    assert max(worst) <= 1, worst


@pytest.mark.parametrize("rows,cols", [(17, 33), (30, 24), (50, 300), (90, 70), (79, 155), (110, 600), (279, 314), (400, 1024), (1800, 500), (830, 2300)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_orthogonalize_at_most(compute, rows, cols, kind):
    """Two and three levels of singular values and one for all: at most 2^-7 of the
    result's norm; permutations and a few elements, whose roundings average out over
    nothing: at most 2^-5."""
    m = min(rows, cols)
    g = gen(rows * cols)
    u, v = (torch.linalg.qr(torch.randn(n, m, generator=g, device="cuda", dtype=torch.float64))[0] for n in (rows, cols))
    i = torch.arange(m, device="cuda", dtype=torch.float64)
    grads, limits = [], []
    for part in (1 / m, 0.03, 0.1, 0.2, 0.4, 0.7, 1.0):
        for floor in (0.3, 0.1, 0.01, 1e-4):
            for middle in (floor, math.sqrt(floor)):
                s = torch.where(i < max(1, int(part * m)), 1.0, torch.where(i < 2 * int(part * m), middle, floor))
                grads.append(((u * s) @ v.T).to(TYPES[kind]).contiguous())
                limits.append(2.0 ** -7)
    for few in (m, m, m, 1, 2, 3, 5, 8, 12, 12):
        x = torch.zeros(rows, cols, device="cuda")
        x[torch.randperm(rows, generator=g, device="cuda")[:few], torch.randperm(cols, generator=g, device="cuda")[:few]] = \
            randn(g, few).sign() * (torch.exp(randn(g, few)) if len(grads) % 2 else 1)
        grads.append(x.to(TYPES[kind]).contiguous())
        limits.append(2.0 ** -5)
    for _ in range(20):
        x = torch.zeros(rows, cols, device="cuda")
        at = torch.randint(0, rows, (12,), generator=g, device="cuda"), torch.randint(0, cols, (12,), generator=g, device="cuda")
        x[at] = randn(g, 12)
        grads.append(x.to(TYPES[kind]).contiguous())
        limits.append(2.0 ** -5)
    for got, grad, limit in zip(orthogonalized(compute, grads, kind), grads, limits):
        want = ref.orthogonalize(grad)
        off, own, size = (float(v.norm()) for v in (got.double() - want, want.bfloat16().double() - want, want))
        assert off <= own + limit * size, (off / size, own / size, limit)


def test_orthogonalize_structures(compute):
    """One large element, equal rows, one direction, an orthogonal matrix, columns of very different sizes."""
    g = gen(5)
    m = randn(g, 160, 224)
    spike = m.clone()
    spike[3, 5] = 1e6
    q = torch.linalg.qr(torch.randn(224, 160, generator=g, device="cuda", dtype=torch.float64))[0].T.float().contiguous()
    cases = [spike, m[:1].repeat(160, 1), randn(g, 160, 1) @ randn(g, 1, 224), q, m * torch.exp(3 * randn(g, 1, 224)), torch.eye(160, 224, device="cuda")]
    for got, grad in zip(orthogonalized(compute, cases), cases):
        near(got, grad)


def test_orthogonalize_zeros_and_padding(compute):
    g = gen(6)
    m = randn(g, 200, 300)
    m[190:], m[:, 290:] = 0, 0
    zero = torch.zeros(200, 300, device="cuda")
    for t in (False, True):
        a, b = orthogonalized(compute, [(v.T if t else v).contiguous() for v in (m, zero)])
        a, b = (a.T, b.T) if t else (a, b)
        assert not bool(a[190:].any()) and not bool(a[:, 290:].any()) and not bool(b.any())
        near(a, m)
        alone = orthogonalized(compute, [(m[:190, :290].T if t else m[:190, :290]).contiguous()])[0]
        near(alone.T if t else alone, m[:190, :290])


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 65537), (3, 3, 70001), (1, 70001, 3), (2, 40, 131077), (1, 200003, 33), (1, 64, 1 << 20),
                                             (2, 1 << 18, 300)])
def test_orthogonalize_long_sides(compute, count, rows, cols):
    """Sums along a long side are as near as others: what they leave stays below the result's own rounding."""
    grads = [randn(gen(rows + i), rows, cols) for i in range(count)]
    for got, grad in zip(orthogonalized(compute, grads), grads):
        near(got, grad)
        want = ref.orthogonalize(grad)
        assert float((got.double() - want).norm()) <= math.sqrt(2) * float((want.bfloat16().double() - want).norm())


def test_orthogonalize_the_longest_vector(compute):
    """One row of 2^26 and some: its length goes through the polynomial, its direction stays."""
    n = (1 << 26) + 3
    grad = randn(gen(17), 1, n)
    got = orthogonalized(compute, [grad])[0].double()
    unit, length = grad.double() / grad.double().norm(), 1.0
    for _ in range(5):
        a, b, c = ref.step_of(ref.COEFFICIENTS, 0)
        length = a * length + b * length ** 3 + c * length ** 5
    # across the direction: the roundings of the elements; along it, where those average out, what the sums leave
    assert float((got - length * unit).norm()) <= ref.U_BF16 * length
    assert abs(float((got * unit).sum()) - length) <= 2.0 ** -9 * length


def test_orthogonalize_not_finite_stays_with_its_matrix(compute):
    g = gen(7)
    grads = [randn(g, 130, 260) for _ in range(4)]
    clean = [v.clone() for v in orthogonalized(compute, grads)]
    grads[1] = grads[1].clone()
    grads[1][129, 259] = math.nan
    grads[2] = grads[2].clone()
    grads[2][0, 0] = math.inf
    got = orthogonalized(compute, grads)
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[2]).all())
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])


@pytest.mark.parametrize("steps", [0, 1, 2, 5])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(3, 70), (130, 40)])
def test_orthogonalize_not_finite_after_any_steps(compute, steps, kind, rows, cols):
    """A matrix with an infinity or NaN becomes NaN all over, one without does not, however many steps."""
    g = gen(15)
    grads = [randn(g, rows, cols, dtype=TYPES[kind]) for _ in range(6)]
    for m, v in zip(grads[1:], (math.nan, math.inf, -math.inf)):
        m[rows // 2, cols // 3] = v
    grads[4] *= 1e38 if kind == "fp32" else 2.0 ** 120  # (in fp32 a few of the larger matrix's are infinite then)
    grads[5] *= 1e37  # its squares leave fp32, as may its norm
    finite = [bool(torch.isfinite(m).all()) for m in grads]
    assert finite[0] and finite[5] and not any(finite[1:4])
    for got, grad, whole in zip(orthogonalized(compute, grads, kind, steps=steps), grads, finite):
        if whole:
            near(got, grad, steps=steps)
        else:
            assert bool(torch.isnan(got).all())


def test_orthogonalize_many(compute):
    """More matrices than one launch takes, the same bits as one by one, every time."""
    grads = gradients(gen(8), 300, 24, 40, "bf16")
    got = orthogonalized(compute, grads, "bf16")
    again = orthogonalized(compute, grads, "bf16")
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i in (0, 1, 127, 128, 129, 255, 256, 299):
        assert torch.equal(orthogonalized(compute, [grads[i]], "bf16")[0], got[i])
        near(got[i], grads[i])


# -------------------------------------------------------- used as programs do

def test_graph_and_streams(compute):
    """One graph of every call, replayed with new inputs, while another stream runs the same calls eagerly."""
    t, e, k, h = 50, 16, 2, 64
    r = tide.Router(e, k, renormalize=True)

    class Job:
        def __init__(self, seed):
            g = gen(seed)
            self.logits, self.x = randn(g, t, e), randn(g, t, h, dtype=torch.bfloat16)
            self.ids, self.slots = (torch.empty(t, k, dtype=torch.int32, device="cuda") for _ in range(2))
            self.w, self.dw = (torch.empty(t, k, device="cuda") for _ in range(2))
            self.offsets = torch.empty(e + 1, dtype=torch.int32, device="cuda")
            self.rows, self.drows = (torch.empty(t * k, h, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.y, self.o = torch.empty_like(self.x), torch.empty_like(self.x)
            self.dlogits = torch.empty_like(self.logits)
            self.ws = torch.empty(tide.orthogonalize_workspace_bytes(1, t, h), dtype=torch.uint8, device="cuda")

        def run(self, s):
            compute.route(r, t, self.logits, self.ids, self.w, stream=s)
            compute.expert_slots(t, k, e, self.ids, self.slots, self.offsets, 0, workspace_bytes=0, stream=s)
            compute.expert_gather(t, h, k, self.x, self.slots, self.rows, t * k, stream=s)
            compute.expert_combine(t, h, k, self.rows, t * k, self.slots, self.w, self.y, stream=s)
            compute.expert_combine_backward(t, h, k, self.y, self.rows, t * k, self.slots, self.w, self.drows, self.dw, stream=s)
            compute.route_backward(r, t, self.logits, self.ids, self.dw, self.dlogits, stream=s)
            compute.orthogonalize(t, h, [self.y], [self.o], self.ws, src_type="bf16", stream=s)

        def results(self):
            return [v.clone() for v in (self.ids, self.w, self.slots, self.offsets, self.rows, self.y, self.drows, self.dw, self.dlogits, self.o)]

    a, b = Job(1), Job(2)
    a.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want_a = a.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(torch.cuda.current_stream())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(side)
    side.synchronize()
    want_b = b.results()
    for _ in range(5):
        graph.replay()
        b.run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), want_a))
    assert all(torch.equal(x, y) for x, y in zip(b.results(), want_b))
    a.logits.copy_(b.logits), a.x.copy_(b.x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), want_b))


def test_expert_layer_step(compute):
    """Routing, experts' gated blocks on their tokens, and back: a whole layer's forward and backward pass against 64 bits."""
    t, e, k, hidden, ffn = 200, 6, 2, 128, 64
    g = gen(9)
    x, logits = randn(g, t, hidden, dtype=torch.bfloat16), randn(g, t, e)
    wg, wu = (randn(g, e, ffn, hidden, scale=hidden ** -0.5, dtype=torch.bfloat16) for _ in range(2))
    dy = randn(g, t, ffn, dtype=torch.bfloat16)
    r = tide.Router(e, k, renormalize=True)
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    ids, slots, w, dw = new(t, k, dtype=torch.int32), new(t, k, dtype=torch.int32), new(t, k, dtype=torch.float32), new(t, k, dtype=torch.float32)
    offsets = new(e + 1, dtype=torch.int32)
    rows, h, y = new(t * k, hidden), new(t * k, ffn), new(t, ffn)
    compute.route(r, t, logits, ids, w)
    compute.expert_slots(t, k, e, ids, slots, offsets, 0, workspace_bytes=0)
    compute.expert_gather(t, hidden, k, x, slots, rows, t * k)
    at = offsets.tolist()
    for i in range(e):
        m = at[i + 1] - at[i]
        if m:
            compute.gated_forward(m, hidden, ffn, rows[at[i]:], wg[i], wu[i], h[at[i]:])
    compute.expert_combine(t, ffn, k, h, t * k, slots, w, y)
    dh, drows, dx, dlogits = new(t * k, ffn), new(t * k, hidden), new(t, hidden), torch.empty_like(logits)
    dwg, dwu = torch.zeros_like(wg), torch.zeros_like(wu)
    compute.expert_combine_backward(t, ffn, k, dy, h, t * k, slots, w, dh, dw)
    for i in range(e):
        m = at[i + 1] - at[i]
        if m:
            ws = new(tide.gated_workspace_bytes(m, hidden, ffn), dtype=torch.uint8)
            compute.gated_backward(m, hidden, ffn, dh[at[i]:], rows[at[i]:], wg[i], wu[i], drows[at[i]:], dwg[i], dwu[i], ws)
    compute.expert_combine(t, hidden, k, drows, t * k, slots, None, dx)
    compute.route_backward(r, t, logits, ids, dw, dlogits)
    outs = [new(ffn, hidden) for _ in range(2 * e)]
    ws = new(tide.orthogonalize_workspace_bytes(2 * e, ffn, hidden), dtype=torch.uint8)
    compute.orthogonalize(ffn, hidden, [*dwg, *dwu], outs, ws, src_type="bf16")
    compute.check_device()
    # the same in 64 bits, by autograd
    leaves = [v.double().requires_grad_(True) for v in (x, logits, wg, wu)]
    lx, ll, lg, lu = leaves
    s = torch.softmax(ll, 1).gather(1, ids.long())
    s = s / s.sum(1, keepdim=True)
    want_y = sum((s * (ids == q)).sum(1, keepdim=True) * (ffn_reference.act(lx @ lg[q].T, "silu") * (lx @ lu[q].T)) for q in range(e))
    grads = torch.autograd.grad((want_y * dy.double()).sum(), leaves)
    # each result has passed a few roundings to bf16 (h, dh, dG and dU, the rows' gradients), 2^-8 of what is rounded at most
    for got, want, roundings in ((y, want_y, 2), (dx, grads[0], 4), (dlogits, grads[1], 3), (dwg, grads[2], 3), (dwu, grads[3], 3)):
        assert float((got.double() - want.detach()).norm()) <= roundings * ref.U_BF16 * float(want.detach().norm())
    for o, grad in zip(outs, [*dwg, *dwu]):
        near(o, grad)


@pytest.mark.parametrize("count,rows,cols", [(1, 100, 200), (1, 704, 256), (3, 700, 1100), (1, 1500, 4000), (100, 300, 600)])
def test_orthogonalize_waits_that_run_out_are_reported(count, rows, cols):
    """Nothing arrives, or one warp of each CTA gives up: the call ends, is reported, and the next one is right."""
    grads = gradients(gen(count), count, rows, cols, "fp32")
    with tide.Compute() as c:
        want = [v.clone() for v in orthogonalized(c, grads)]
        c.check_device()
        for hook in (c.set_test_stall, c.set_test_late_warp):
            hook(1_000_000)
            orthogonalized(c, grads)
            with pytest.raises(tide.TideError) as e:
                c.check_device()
            assert e.value.status == tide.TIDE_ERR_TIMEOUT
            hook(0)
            assert all(torch.equal(a, b) for a, b in zip(orthogonalized(c, grads), want))
            c.check_device()


def test_expert_layer_example():
    """The example runs, its first step's mean gradients are the definition's, and its updates their orthogonal factors."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import expert_layer as ex

    ranks, tokens, experts, topk, hidden, ffn = 2, 70, 5, 2, 128, 96
    layer = ex.Layer(ranks, experts, topk, hidden, ffn)
    inputs, targets = ex.problem(layer, tokens, 1)
    work = ex.Pass(layer, tokens)
    with tide.Compute() as c:
        loss = ex.step(layer, c, work, inputs, targets, 0.0)  # the parameters stay as they were
        leaves = [p.double().requires_grad_(True) for p in layer.params]
        total = 0.0
        for r in range(ranks):
            logits = inputs[r].double() @ leaves[0].T
            ids, _ = ref.route(logits.detach().float(), topk)
            share = torch.softmax(logits, 1).gather(1, ids)
            share = share / share.sum(1, keepdim=True)
            x, y = inputs[r].double(), 0.0
            for e in range(experts):
                gate, up, down = layer.expert(leaves, e)
                mine = (share * (ids == e)).sum(1, keepdim=True)
                y = y + mine * ((ffn_reference.act(x @ gate.T, "silu") * (x @ up.T)) @ down.T)
            total = total + ((y - targets[r].double()) ** 2).mean() / ranks
        assert abs(loss - float(total.detach())) <= 4 * ref.U_BF16 * float(total.detach())
        grads = torch.autograd.grad(total, leaves)
        # y - target, dz, h, z, dh, dG and dU, and the gradients themselves have been rounded to bf16, the mean once more
        for got, want in zip(layer.whole, grads):
            assert float((got.double() - want).norm()) <= 6 * ref.U_BF16 * float(want.norm())
        for p, (update, grad) in enumerate(zip(layer.updates, layer.whole)):
            if p:
                near(update, grad)
        losses = [ex.step(layer, c, work, inputs, targets, 0.02) for _ in range(2)]
        assert all(math.isfinite(v) for v in losses)


# --------------------------------------------------- past 32-bit offsets

def test_route_past_32_bit_offsets(compute):
    """The last tokens of 2.1 million among 1024 experts choose as they do alone, forward and back."""
    t, e, k, some = (1 << 21) + 77, 1024, 4, 300
    g = gen(40)
    r = tide.Router(e, k)
    logits = torch.empty(t, e, dtype=torch.bfloat16, device="cuda")
    for part in logits.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    ids, w = torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(t, k, device="cuda")
    compute.route(r, t, logits, ids, w, logits_type="bf16")
    last = logits[-some:].clone()
    check_route(compute, dict(experts=e, topk=k), last, None, "bf16")
    ids1, w1 = torch.empty(some, k, dtype=torch.int32, device="cuda"), torch.empty(some, k, device="cuda")
    compute.route(r, some, last, ids1, w1, logits_type="bf16")
    assert torch.equal(ids[-some:], ids1) and torch.equal(w[-some:], w1)
    dlogits, alone = torch.empty_like(logits), torch.empty_like(last)
    compute.route_backward(r, t, logits, ids, w, dlogits, logits_type="bf16")
    compute.route_backward(r, some, last, ids1, w1, alone, logits_type="bf16")
    assert torch.equal(dlogits[-some:], alone)


def test_rows_past_32_bit_offsets(compute):
    """36,000 tokens of 8192 to 8 experts each, 2.4 billion elements, there and back."""
    t, h, k = 36000, 8192, 8
    g = gen(41)
    x = torch.randn(t, h, generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, 64, (t, k), generator=g, device="cuda", dtype=torch.int32)
    slots, offsets = torch.empty_like(ids), torch.empty(65, dtype=torch.int32, device="cuda")
    ws = torch.empty(tide.expert_slots_workspace_bytes(t, k, 64), dtype=torch.uint8, device="cuda")
    compute.expert_slots(t, k, 64, ids, slots, offsets, ws)
    rows = torch.empty(t * k, h, dtype=torch.bfloat16, device="cuda")
    compute.expert_gather(t, h, k, x, slots, rows, t * k)
    for i in (0, t // 2, t - 1):
        assert torch.equal(rows[slots[i].long()], x[i].expand(k, h))
    y = torch.empty_like(x)
    w = torch.rand(t, k, generator=g, device="cuda")
    compute.expert_combine(t, h, k, rows, t * k, slots, w, y)
    drows, dw = torch.empty_like(rows), torch.empty_like(w)
    compute.expert_combine_backward(t, h, k, x, rows, t * k, slots, w, drows, dw)
    for part in (slice(0, 50), slice(t - 50, t)):
        at = slots[part].reshape(-1).long()
        few = torch.arange(at.numel(), device="cuda", dtype=torch.int32).view(-1, k)
        want, bound = ref.combine(rows[at], few, w[part])
        close(y[part], want, bound)
        each, each_bound, want_dw, dw_bound = ref.combine_backward(x[part], rows[at], few, w[part])
        close(drows[at].view(-1, k, h), each, each_bound)
        close(dw[part], want_dw, dw_bound)


def test_orthogonalize_past_32_bit_offsets(compute):
    """600 matrices of 1000 x 4000 in one call: 2.4 billion elements in each plane."""
    count, rows, cols = 600, 1000, 4000
    g = gen(42)
    grads = torch.empty(count, rows, cols, dtype=torch.bfloat16, device="cuda")
    for part in grads.split(50):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    outs = torch.empty_like(grads)
    ws = torch.empty(tide.orthogonalize_workspace_bytes(count, rows, cols), dtype=torch.uint8, device="cuda")
    compute.orthogonalize(rows, cols, list(grads), list(outs), ws, src_type="bf16")
    del ws
    for i in (0, 127, 128, count - 1):
        near(outs[i], grads[i])
