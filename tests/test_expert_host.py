"""The expert layer's operators without a GPU: refusals, sizes, and the formulas
the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import expert_reference as ref
import layout_aware_collectives_gb300 as tide
from test_compute_host import A, BAD, MIS, refused


@pytest.fixture
def compute():
    with tide.Compute() as c:
        yield c


def test_router_refuses(compute):
    def call(router, tokens=4, **kw):
        return compute.route(router, tokens, A, A, A, **kw)

    ok = dict(experts=8, topk=2)
    for bad in (dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=9), dict(experts=64, topk=17), dict(score=2),
                dict(groups=0), dict(groups=3), dict(groups=2, top_groups=3), dict(groups=2, top_groups=0),
                dict(groups=4, top_groups=1, topk=3), dict(group_best=0), dict(group_best=3), dict(experts=66, groups=33)):
        refused(BAD, call, tide.Router(**{**ok, **bad}))
    r = tide.Router(**ok)
    refused(BAD, call, None, ld_logits=8)
    refused(BAD, call, r, tokens=-1)
    refused(BAD, call, r, tokens=1 << 31)
    refused(BAD, call, r, ld_logits=7)
    refused(BAD, call, r, logits_type=5)
    refused(MIS, call, r, bias=A + 2)
    with pytest.raises(ValueError):
        call(r, logits_type="fp64")
    with pytest.raises(ValueError):
        tide.Router(8, 2, score="argmax")
    for i, v, st in ((0, 0, BAD), (1, 0, BAD), (2, 0, BAD), (0, A + 2, MIS), (1, A + 1, MIS), (2, A + 2, MIS)):
        args = [A, A, A]
        args[i] = v
        refused(st, compute.route, r, 4, *args)
    compute.route(r, 0, 0, 0, 0)  # nothing to do, no device touched
    for i, v, st in ((0, 0, BAD), (1, 0, BAD), (2, 0, BAD), (3, 0, BAD), (1, A + 2, MIS), (3, A + 2, MIS)):
        args = [A, A, A, A]
        args[i] = v
        refused(st, compute.route_backward, r, 4, *args)
    refused(BAD, compute.route_backward, r, 4, A, A, A, A, ld_dlogits=7)
    compute.route_backward(r, 0, 0, 0, 0, 0)


def test_slots_refuse(compute):
    n = tide.expert_slots_workspace_bytes(5000, 8, 128)
    assert n > 0 and tide.expert_slots_workspace_bytes(37, 8, 128) == 0
    ok = [5000, 8, 128, A, A, A, A]
    kw = dict(workspace_bytes=n)
    for i, v, st in ((0, -1, BAD), (0, 1 << 28, BAD), (1, 0, BAD), (1, 1025, BAD), (2, 0, BAD), (2, 1025, BAD), (3, 0, BAD),
                     (4, 0, BAD), (5, 0, BAD), (6, 0, BAD), (3, A + 2, MIS), (6, A + 8, MIS)):
        bad = list(ok)
        bad[i] = v
        refused(st, compute.expert_slots, *bad, **kw)
    refused(BAD, compute.expert_slots, *ok, workspace_bytes=n - 1)
    for bad in ((-1, 8, 128), (4, 0, 128), (4, 8, 0), (4, 8, 2000)):
        with pytest.raises(tide.TideError):
            tide.expert_slots_workspace_bytes(*bad)


def test_rows_refuse(compute):
    ok = [4, 64, 2, A, A, A, 8]
    for f, gather in ((compute.expert_gather, True), (lambda t, h, k, r, s, y, n, **kw: compute.expert_combine(t, h, k, r, n, s, A, y, **kw), False)):
        for i, v, st in ((0, -1, BAD), (1, -1, BAD), (2, 0, BAD), (2, 2000, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (6, -1, BAD),
                         (3, A + 2, MIS), (4, A + 2, MIS), (5, A + 8, MIS)):
            bad = list(ok)
            bad[i] = v
            refused(st, f, *bad)
        refused(BAD, f, *ok, ld_rows=63)
        refused(BAD, f, *ok, **{"ld_x" if gather else "ld_y": 63})
        f(0, 64, 2, 0, 0, 0, 0)
        f(4, 0, 2, 0, A, 0, 8)
    refused(MIS, compute.expert_combine, 4, 64, 2, A, 8, A, A + 2, A)
    good = [4, 64, 2, A, A, 8, A, A, A, A]
    for i, v, st in ((3, 0, BAD), (4, 0, BAD), (6, 0, BAD), (7, A + 2, MIS), (8, A + 2, MIS), (9, A + 2, MIS)):
        bad = list(good)
        bad[i] = v
        refused(st, compute.expert_combine_backward, *bad)
    for ld in ("ld_dy", "ld_rows", "ld_drows"):
        refused(BAD, compute.expert_combine_backward, *good, **{ld: 63})
    compute.expert_combine_backward(4, 64, 2, A, 0, 8, A, A, None, None)
    compute.expert_combine_backward(0, 64, 2, 0, 0, 0, 0, 0, 0, 0)


def test_orthogonalize_refuses(compute):
    n = tide.orthogonalize_workspace_bytes(2, 8, 16)

    def call(rows=8, cols=16, src=(A, A), dst=(A, A), workspace=A, **kw):
        compute.orthogonalize(rows, cols, src, dst, workspace, **{"workspace_bytes": n, **kw})

    for bad in (dict(rows=-1), dict(cols=1 << 31), dict(rows=1 << 20, cols=1 << 20), dict(src=(A, 0)), dict(dst=(0, A)), dict(ld_src=15),
                dict(ld_dst=15), dict(steps=-1), dict(steps=17), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan),
                dict(workspace=0), dict(workspace_bytes=n - 1), dict(src_type=3), dict(coefficients=(math.nan, 0, 0)),
                dict(coefficients=(1e6, 0, 0)), dict(coefficients=(8, 0, 0), steps=6), dict(coefficients=(1, 1, math.inf)),
                dict(steps=4, coefficients=(8.0, -22.0, 16.0, 4.0, -3.0, 0.6, 3.8, -2.8, 0.55, 3.0, -2.2, 0.45))):
        refused(BAD, call, **bad)
    for bad in (dict(src=(A, A + 2)), dict(src=(A, A + 1), src_type="bf16"), dict(dst=(A + 1, A)), dict(workspace=A + 128 + 8)):
        refused(MIS, call, **bad)
    with pytest.raises(ValueError):
        call(src=(A,))
    with pytest.raises(ValueError):
        call(coefficients=(1, 2, 3, 4))
    call(src=(), dst=(), workspace=0, workspace_bytes=0)
    call(rows=0, workspace=0, workspace_bytes=0, src=(0, 0), dst=(0, 0))
    for bad in ((-1, 4, 4), (1, -4, 4), (1 << 38, 4, 4), (1 << 31, 1, 1), (1, (1 << 30) + 1, 1), (1, 1, (1 << 31) - 1)):
        with pytest.raises(tide.TideError):
            tide.orthogonalize_workspace_bytes(*bad)


def test_null_handle_refused():
    lib = tide.tide._lib
    r = tide.Router(8, 2)
    p = ctypes.addressof(r.struct)
    assert lib.tide_route(None, 1, p, 1, A, 8, None, A, A, None) == BAD
    assert lib.tide_route_backward(None, 1, p, 1, A, 8, A, A, A, 8, None) == BAD
    assert lib.tide_expert_slots(None, 1, 1, 8, A, A, A, A, 0, None) == BAD
    assert lib.tide_expert_gather(None, 1, 8, 1, A, 8, A, A, 1, 8, None) == BAD
    assert lib.tide_expert_combine(None, 1, 8, 1, A, 1, 8, A, A, A, 8, None) == BAD
    assert lib.tide_expert_combine_backward(None, 1, 8, 1, A, 8, A, 1, 8, A, A, A, 8, A, None) == BAD
    assert lib.tide_orthogonalize(None, 0, 1, 1, 1, None, 1, None, 1, 5, None, 0.0, None, 0, None) == BAD
    assert lib.tide_expert_slots_workspace(1, 1, 1, None) == BAD
    assert lib.tide_orthogonalize_workspace(1, 1, 1, None) == BAD
    assert ctypes.sizeof(tide.tide.RouterStruct) == 32


def differences(f, at, step):
    out = torch.zeros_like(at)
    for i in range(at.numel()):
        side = []
        for s in (step, -step):
            moved = at.clone()
            moved.view(-1)[i] += s
            side.append(f(moved))
        out.view(-1)[i] = (side[0] - side[1]) / (2 * step)
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_formulas_against_differences(score, renormalize):
    """The 64-bit gradients are the differences of the 64-bit weights."""
    g = torch.Generator().manual_seed(5)
    l = torch.randn(3, 7, generator=g, dtype=torch.float64)
    dw = torch.randn(3, 2, generator=g, dtype=torch.float64)
    ids, _ = ref.route(l, 2, score, renormalize=renormalize, scale=2.5)

    def loss(moved):
        w = ref.scores(moved, score).gather(1, ids)
        return float((dw * (w / w.sum(1, keepdim=True) if renormalize else w)).sum() * 2.5)

    got, _ = ref.route_backward(l, ids, dw, score, renormalize, 2.5)
    # central difference: error ~ step^2 f''' + 2^-53 / step
    assert float((differences(loss, l, 1e-6) - got).abs().max()) < 1e-8


def test_combine_formulas_against_differences():
    g = torch.Generator().manual_seed(6)
    rows, w, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((6, 4), (3, 2), (3, 4)))
    at = torch.tensor([[0, 3], [5, 1], [2, -1]], dtype=torch.int32)
    drows, _, dw, _ = ref.combine_backward(dy, rows, at, w)
    assert float((differences(lambda v: float((ref.combine(rows, at, v)[0] * dy).sum()), w, 1e-6) - dw).abs().max()) < 1e-8
    by = differences(lambda v: float((ref.combine(v, at, w)[0] * dy).sum()), rows, 1e-6)
    for t in range(3):
        for j in range(2):
            if at[t, j] >= 0:
                assert float((by[at[t, j]] - drows[t, j]).abs().max()) < 1e-8


def test_orthogonalize_definition():
    """Singular vectors stay, singular values go through the polynomial."""
    g = torch.Generator().manual_seed(7)
    for shape in ((5, 9), (9, 5), (6, 6)):
        m = torch.randn(*shape, generator=g, dtype=torch.float64)
        u, s, v = torch.linalg.svd(m, full_matrices=False)
        s = s / (s.norm() + 1e-7)
        for i in range(5):
            a, b, c = ref.step_of(ref.COEFFICIENTS, i)
            s = a * s + b * s ** 3 + c * s ** 5
        assert float((ref.orthogonalize(m) - u @ torch.diag(s) @ v).abs().max()) < 1e-10
        assert 0.6 < float(s.min()) and float(s.max()) < 1.25


def test_published_writes_pass_the_proxies_before_the_release():
    """What a thread has written reaches other CTAs' copies by tensor maps only if
    the proxies' fence lies between the writes and the release that carries them."""
    import os

    csrc = os.path.join(os.path.dirname(tide.__file__), "csrc")
    with open(os.path.join(csrc, "tc_device.cuh")) as f:
        body = f.read().split("void publish() {")[1].split("\n}")[0]
    assert 0 <= body.find("fence.proxy.async;") < body.find("fence.acq_rel.cluster;")


@pytest.fixture
def calls(monkeypatch):
    """What reaches the library's entries of an expert layer, by name."""
    class Library:
        def __init__(self, lib):
            self.lib, self.made = lib, {}

        def __getattr__(self, name):
            if name not in ("tide_route", "tide_route_backward", "tide_orthogonalize", "tide_expert_slots", "tide_expert_gather",
                            "tide_expert_combine", "tide_expert_combine_backward"):
                return getattr(self.lib, name)
            return lambda *args: self.made.__setitem__(name, args) or 0

    library = Library(tide.tide._lib)
    monkeypatch.setattr(tide.tide, "_lib", library)
    return library.made


def test_elements_are_read_as_what_they_are(compute, calls):
    """bf16 logits and gradients without a word about their type are bf16: as fp32
    they would be read to twice their length."""
    r = tide.Router(8, 2)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for dtype, code, name in ((torch.bfloat16, 0, "bf16"), (torch.float32, 1, "fp32")):
        logits = torch.zeros(4, 8, dtype=dtype)
        for kw in ({}, dict(logits_type=name), dict(logits_type=code)):
            compute.route(r, 4, logits, ids, w, **kw)
            assert calls.pop("tide_route")[3] == code
            compute.route_backward(r, 4, logits, ids, w, torch.zeros_like(logits), **kw)
            assert calls.pop("tide_route_backward")[3] == code
        m = [torch.zeros(4, 8, dtype=dtype) for _ in range(2)]
        out = [torch.zeros(4, 8, dtype=torch.bfloat16) for _ in range(2)]
        for src in (m, tide.PointerTable(m)):
            for kw in ({}, dict(src_type=name)):
                compute.orthogonalize(4, 8, src, out, A, workspace_bytes=1 << 20, **kw)
                assert calls.pop("tide_orthogonalize")[4] == code
    compute.route(r, 4, A, ids, w)  # an address says nothing
    assert calls.pop("tide_route")[3] == 1


def test_elements_of_other_types_are_refused(compute, calls):
    r = tide.Router(8, 2)
    z = lambda dtype, *s: torch.zeros(*(s or (4, 2)), dtype=dtype)  # noqa: E731
    i32, i64, f32, f64, bf16, f16 = torch.int32, torch.int64, torch.float32, torch.float64, torch.bfloat16, torch.float16

    def refuses(f, good, bad, **kw):
        f(*good, **kw)
        calls.clear()
        for at, dtypes in bad.items():
            for dtype in dtypes:
                args = list(good)
                args[at] = z(dtype)
                with pytest.raises(TypeError):
                    f(*args, **kw)
        assert not calls

    refuses(compute.route, [r, 4, z(f32), z(i32), z(f32)], {2: (f64, f16, i32), 3: (i64, f32), 4: (bf16, f64)})
    refuses(compute.route, [r, 4, z(f32), z(i32), z(f32), z(f32)], {5: (bf16, f64)})
    refuses(compute.route, [r, 4, z(f32), z(i32), z(f32)], {2: (bf16,)}, logits_type="fp32")
    refuses(compute.route_backward, [r, 4, z(f32), z(i32), z(f32), z(f32)], {2: (bf16, f64), 3: (i64,), 4: (bf16,), 5: (bf16, f64)})
    refuses(compute.expert_slots, [4, 2, 8, z(i32), z(i32), z(i32), A], {3: (i64,), 4: (i64,), 5: (i64, f32)}, workspace_bytes=0)
    refuses(compute.expert_gather, [4, 2, 2, z(bf16), z(i32), z(bf16), 8], {3: (f32, f16), 4: (i64,), 5: (f32,)})
    refuses(compute.expert_combine, [4, 2, 2, z(bf16), 8, z(i32), z(f32), z(bf16)], {3: (f32,), 5: (i64,), 6: (bf16,), 7: (f32,)})
    refuses(compute.expert_combine_backward, [4, 2, 2, z(bf16), z(bf16), 8, z(i32), z(f32), z(bf16), z(f32)],
            {3: (f32,), 4: (f32,), 6: (i64,), 7: (bf16,), 8: (f32,), 9: (bf16,)})
    for src, dst, kw in (([z(f64)], [z(bf16)], {}), ([z(f32), z(bf16)], [z(bf16)] * 2, {}), ([z(f32)], [z(f32)], {}),
                         ([z(bf16)], [z(bf16)], dict(src_type="fp32")), ([z(f32)], [z(bf16)], dict(src_type="bf16"))):
        with pytest.raises(TypeError):
            compute.orthogonalize(4, 2, src, dst, A, workspace_bytes=1 << 20, **kw)
    assert not calls


def test_orthogonalize_sizes_of_long_and_short_sides():
    """Sides up to 2^30, of which one is up to 2^17; a workspace that holds what long sides' sums take."""
    for ok in ((1, 1 << 17, 1 << 17), (1, 1 << 30, 3), (1, 3, 1 << 30), (1, 1 << 21, 1 << 17)):
        assert tide.orthogonalize_workspace_bytes(*ok) > 0
    for bad in ((1, (1 << 17) + 1, (1 << 17) + 1), (1, 1 << 18, 1 << 18)):
        with pytest.raises(tide.TideError):
            tide.orthogonalize_workspace_bytes(*bad)
    m, n = 100, 65536
    planes = 4 * m * n * 2 + 3 * m * 128 * 2 + 3 * m * 4
    assert planes <= tide.orthogonalize_workspace_bytes(1, m, n) < planes + (1 << 16)
    n += 64
    assert tide.orthogonalize_workspace_bytes(1, m, n) >= 4 * m * n * 2 + (3 + 2) * m * 128 * 2 + (3 + 2) * m * 4
