"""Feed-forward operators on the GPU against their 64-bit definitions.

Bounds come from the formats (see ffn_reference); outputs are framed by guard
elements that must stay as they were."""
import math

import pytest

torch = pytest.importorskip("torch")

import ffn_reference as ref  # noqa: E402
import layout_aware_collectives_gb300 as tide  # noqa: E402

pytestmark = pytest.mark.gpu

GUARD = 64


@pytest.fixture(scope="module")
def compute():
    with tide.Compute() as c:
        yield c


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


class Guarded:
    """An output of `rows` rows of `cols` elements, `ld` apart, in a buffer
    filled with a value that nothing may overwrite around it."""

    def __init__(self, rows, cols, ld=None, dtype=torch.bfloat16):
        self.rows, self.cols, self.ld = rows, cols, cols if ld is None else ld
        self.fill = 0x5A
        n = GUARD + max(0, rows - 1) * self.ld + cols + GUARD
        size = torch.empty(0, dtype=dtype).element_size()
        self.bytes = torch.full((n * size,), self.fill, dtype=torch.uint8, device="cuda")
        self.all = self.bytes.view(dtype)
        self.size = size
        self.t = self.all[GUARD:GUARD + max(0, rows - 1) * self.ld + cols]
        self.view = torch.as_strided(self.all, (rows, cols), (self.ld, 1), GUARD)

    def data_ptr(self):
        return self.t.data_ptr()

    def intact(self):
        at = torch.arange(self.all.numel(), device="cuda") - GUARD
        mine = (at >= 0) & (at < (self.rows - 1) * self.ld + self.cols) & (at.remainder(self.ld) < self.cols)
        rest = self.bytes.view(-1, self.size)[~mine]
        return bool((rest == self.fill).all())


def strided(t, ld):
    """A copy of t with rows ld apart."""
    buf = torch.full((t.shape[0], ld), math.nan, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf


def close(got, want, bound):
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside; worst {float((got - want).abs().sub(bound)[bad].max())}"


# ------------------------------------------------------------------- blocks

BLOCK_SHAPES = [(1, 1), (1, 128), (3, 129), (5, 250), (37, 768), (130, 136), (257, 1000), (128, 128), (64, 2049)]


def awkward(g, rows, cols):
    """Values over the whole range: zeros, subnormals, the largest, infinities, NaN, exact block limits."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(
        torch.randint(-120, 120, (rows, 1), generator=g, device="cuda").float())
    flat = v.view(-1)
    for i, s in enumerate((0.0, math.inf, -math.inf, math.nan, 448.0, 449.0, 464.0, 3.3e38, 1e-40, -0.0, 2.0 ** -133)):
        flat[torch.randint(0, flat.numel(), (max(1, flat.numel() // 97),), generator=g, device="cuda")] = s
    if rows > 2:
        v[1] = 0
        v[2, : cols // 2] = 1e-39
    return v.bfloat16()


def same_codes(got, want):
    a, b = got.float(), want.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    a, b = torch.nan_to_num(a), torch.nan_to_num(b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", BLOCK_SHAPES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_store(compute, rows, cols, block_rows, pad):
    g = gen(rows * 1000 + cols)
    for v in (randn(g, rows, cols), awkward(g, rows, cols)):
        codes = Guarded(rows, cols, dtype=torch.float8_e4m3fn)
        scales = Guarded(-(-rows // block_rows), -(-cols // 128), dtype=torch.float32)
        compute.fp8_store(rows, cols, strided(v, cols + pad) if pad else v, codes, scales, block_rows=block_rows,
                          ld_src=cols + pad)
        want_codes, want_scales = ref.blocks_store(v.float().cpu(), block_rows)
        assert torch.equal(scales.view.cpu(), want_scales)
        same_codes(codes.view.cpu(), want_codes)
        assert codes.intact() and scales.intact()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", BLOCK_SHAPES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_restore(compute, rows, cols, block_rows, pad):
    g = gen(rows * 1000 + cols + 1)
    codes = torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    # any scale, not powers of two alone
    scales = torch.randn(-(-rows // block_rows), -(-cols // 128), generator=g, device="cuda").exp()
    dst = Guarded(rows, cols, cols + pad)
    compute.fp8_restore(rows, cols, codes, scales, dst, block_rows=block_rows, ld_dst=cols + pad)
    want = ref.blocks_value(codes.view(torch.float8_e4m3fn), scales, block_rows).float().bfloat16()
    assert torch.equal(torch.isnan(dst.view), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(dst.view), torch.nan_to_num(want))
    assert dst.intact()


# ------------------------------------------------------------------ products

MATMUL_SHAPES = [(1, 128, 128), (1, 8, 16), (2, 264, 400), (3, 1, 1), (7, 130, 129), (37, 768, 2048), (129, 264, 1040),
                 (250, 704, 256), (300, 520, 144), (33, 100, 300), (513, 1024, 4096),
                 (300, 5000, 272), (64, 136, 8192), (70, 1160, 1296), (300, 5200, 400), (1000, 4864, 160)]


def fp8(g, rows, cols, block_rows, any_scales=False):
    v = torch.randn(rows, cols, generator=g, device="cuda")
    codes = (v * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    shape = -(-rows // block_rows), -(-cols // 128)
    if any_scales:
        return codes, torch.randn(*shape, generator=g, device="cuda").exp()
    return codes, torch.exp2(torch.randint(-9, 10, shape, generator=g, device="cuda").float())


@pytest.mark.parametrize("m,n,k", MATMUL_SHAPES)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("any_scales", [False, True])
def test_matmul(compute, m, n, k, pad, any_scales):
    g = gen(m + n + k)
    (a, sa), (b, sb) = fp8(g, m, k, 1, any_scales), fp8(g, n, k, 128, any_scales)
    out = Guarded(m, n, n + pad)
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out, any_scales=any_scales, ld_out=n + pad)
    close(out.view, *ref.matmul(a, sa, b, sb))
    assert out.intact()


# few tiles and a long contraction: split in two, three and four
@pytest.mark.parametrize("m,n,k", [(1014, 752, 9200), (200, 2368, 7904), (1100, 1000, 3216), (1500, 1288, 2064), (65, 8192, 2176)])
@pytest.mark.parametrize("pad", [0, 8])
def test_matmul_split(compute, m, n, k, pad):
    g = gen(m + n + k)
    (a, sa), (b, sb) = fp8(g, m, k, 1), fp8(g, n, k, 128)
    out = Guarded(m, n, n + pad)
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out, ld_out=n + pad)
    close(out.view, *ref.matmul(a, sa, b, sb))
    assert out.intact()
    first = out.view.clone()
    for _ in range(3):
        compute.fp8_matmul(m, n, k, a, sa, b, sb, out, ld_out=n + pad)
        assert torch.equal(out.view, first)
    sa[m - 1, -1] = 1.5  # no power of two
    a.view(torch.uint8)[3, k - 1] = 0x7F
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out, ld_out=n + pad)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[m - 1], nan[3] = True, True
    assert torch.equal(torch.isnan(out.view), nan) and torch.equal(out.view[:3], first[:3])


def test_matmul_split_wait_that_runs_out_is_reported():
    m, n, k = 1014, 752, 9200
    g = gen(31)
    (a, sa), (b, sb) = fp8(g, m, k, 1), fp8(g, n, k, 128)
    out = Guarded(m, n)
    with tide.Compute() as c:
        c.set_test_stall(1_000_000)
        c.fp8_matmul(m, n, k, a, sa, b, sb, out)
        with pytest.raises(tide.TideError) as e:
            c.check_device()
        assert e.value.status == tide.TIDE_ERR_TIMEOUT
        c.set_test_stall(0)
        c.fp8_matmul(m, n, k, a, sa, b, sb, out)
        c.check_device()
        close(out.view, *ref.matmul(a, sa, b, sb))
        assert out.intact()


@pytest.mark.parametrize("m,n,k", [(3, 264, 512), (300, 5000, 272), (5, 130, 129)])
@pytest.mark.parametrize("bad", [1.5, 0.0, -2.0, math.inf, math.nan, 1e-40])
def test_matmul_scale_that_is_no_power_of_two(compute, m, n, k, bad):
    g = gen(77)
    (a, sa), (b, sb) = fp8(g, m, k, 1), fp8(g, n, k, 128)
    sa[1, 1], sb[1, 0] = bad, bad
    out = Guarded(m, n)
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1], nan[:, 128:256] = True, True
    assert torch.equal(torch.isnan(out.view), nan) and out.intact()


@pytest.mark.parametrize("m,n", [(4, 264), (300, 5000)])
def test_matmul_extreme_scales(compute, m, n):
    """Scales over their whole range; results that fp32 holds keep their value."""
    k = 384
    g = gen(78)
    (a, sa), (b, sb) = fp8(g, m, k, 1), fp8(g, n, k, 128)
    up = torch.randint(0, 2, (m, 1), generator=g, device="cuda").float() * 200 - 100  # 2^-100 or 2^100 a row
    sa, sb = torch.exp2(up).expand(m, 3).contiguous(), torch.exp2(torch.zeros_like(sb))
    out = Guarded(m, n)
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out)
    close(out.view, *ref.matmul(a, sa, b, sb))


def test_matmul_empty_sum(compute):
    out = Guarded(5, 16, 24)
    compute.fp8_matmul(5, 16, 0, 0, 0, 0, 0, out, ld_out=24)
    assert (out.view == 0).all() and out.intact()


def test_matmul_nan_stays_in_its_row_and_column(compute):
    g = gen(5)
    for m, n in ((20, 264), (140, 5000)):
        for any_scales in (False, True):
            (a, sa), (b, sb) = fp8(g, m, 512, 1), fp8(g, n, 512, 128)
            a.view(torch.uint8)[3, 200] = 0x7F
            b.view(torch.uint8)[129, 17] = 0xFF
            out = Guarded(m, n)
            compute.fp8_matmul(m, n, 512, a, sa, b, sb, out, any_scales=any_scales)
            nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
            nan[3], nan[:, 129] = True, True
            assert torch.equal(torch.isnan(out.view), nan)


# --------------------------------------------------------------------- gated

# tokens, hidden, ffn: one token, single columns, ragged and unaligned sizes,
# several tiles each way
GATED_SHAPES = [(1, 256, 704), (1, 8, 8), (3, 1, 1), (5, 250, 130), (16, 128, 128), (17, 264, 136), (37, 2048, 768),
                (129, 72, 1000), (250, 256, 704), (300, 1032, 264), (513, 512, 1408),
                (300, 136, 2568), (20, 4104, 256), (50, 1000, 1400), (60, 264, 4104), (3000, 72, 136)]


def checkpoint(tokens, hidden, ffn, with_x):
    c = {n: Guarded(tokens, ffn, dtype=torch.float8_e4m3fn) for n in ("g8", "u8")}
    c |= {n: Guarded(tokens, -(-ffn // 128), dtype=torch.float32) for n in ("gs", "us")}
    if with_x:
        c["x8"] = Guarded(tokens, hidden, dtype=torch.float8_e4m3fn)
        c["xs"] = Guarded(tokens, -(-hidden // 128), dtype=torch.float32)
    return c, tide.GatedCheckpoint(c["g8"], c["gs"], c["u8"], c["us"], c.get("x8"), c.get("xs"))


def weights(g, hidden, ffn):
    return randn(g, ffn, hidden, scale=hidden ** -0.5), randn(g, ffn, hidden, scale=hidden ** -0.5)


def close_to_stored(codes, scales, want, err):
    """Stored values are within e4m3's rounding (half a step: 2^-4 of the value,
    2^-10 of the scale below its normal range) of values within `err` of want,
    and each scale is the power of two its block's maximum asks for."""
    got = ref.blocks_value(codes, scales, 1)
    j = torch.arange(codes.shape[1], device="cuda") // 128
    close(got, want, err + 2.0 ** -4 * (want.abs() + err) + 2.0 ** -10 * scales.double()[:, j])
    for b in range(scales.shape[1]):
        top = want[:, b * 128:(b + 1) * 128].abs().amax(1)
        off = err[:, b * 128:(b + 1) * 128].amax(1)
        s = scales[:, b].double()
        assert (torch.frexp(scales[:, b])[0] == 0.5).all()
        assert ((top - off <= 448 * s) & ((top + off > 224 * s) | (s <= 2.0 ** -126) | (top == 0))).all()


@pytest.mark.parametrize("tokens,hidden,ffn", GATED_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("keep", ["none", "pre", "all"])
def test_gated_forward(compute, tokens, hidden, ffn, kind, keep):
    g = gen(tokens + hidden + ffn)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, hidden, ffn, keep == "all") if keep != "none" else ({}, None)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, activation=kind, checkpoint=ck)
    want, gg, uu = ref.gated_forward(x, wg, wu, kind)
    bh, eg, eu = ref.gated_forward_bound(x, wg, wu, kind)
    close(h.view, want, bh)
    assert h.intact() and all(b.intact() for b in bufs.values())
    if ck:
        close_to_stored(bufs["g8"].view, bufs["gs"].view, gg, eg)
        close_to_stored(bufs["u8"].view, bufs["us"].view, uu, eu)
    if keep == "all":
        codes, scales = ref.blocks_store(x.float().cpu(), 1)
        assert torch.equal(bufs["xs"].view.cpu(), scales)
        same_codes(bufs["x8"].view.cpu(), codes)


# few tiles and a long contraction: split in two, three and four
SPLIT_SHAPES = [(1014, 9200, 752), (200, 7904, 2368), (100, 8200, 1000), (1021, 2048, 768), (300, 1544, 136)]


@pytest.mark.parametrize("tokens,hidden,ffn", SPLIT_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("keep", ["none", "pre"])
def test_gated_forward_split(compute, tokens, hidden, ffn, kind, keep):
    test_gated_forward(compute, tokens, hidden, ffn, kind, keep)


@pytest.mark.parametrize("tokens,hidden,ffn", SPLIT_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_backward_split(compute, tokens, hidden, ffn, kind):
    test_gated_backward_recomputed(compute, tokens, hidden, ffn, kind, True)


def test_gated_split_same_results_every_time(compute):
    """In the parts' order each time, with a checkpoint or without one."""
    tokens, hidden, ffn = 200, 7904, 2368
    g = gen(22)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    h = Guarded(tokens, ffn, ffn + 8)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, ld_h=ffn + 8)
    first, grads = h.view.clone(), [t.clone() for t in run_backward(compute, tokens, hidden, ffn, "silu", dh, x, wg, wu)]
    for _ in range(5):
        bufs, ck = checkpoint(tokens, hidden, ffn, False)
        compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck, ld_h=ffn + 8)
        assert torch.equal(h.view, first) and h.intact() and all(b.intact() for b in bufs.values())
        for a, b in zip(grads, run_backward(compute, tokens, hidden, ffn, "silu", dh, x, wg, wu)):
            assert torch.equal(a, b)


def test_gated_split_wait_that_runs_out_is_reported():
    tokens, hidden, ffn = 200, 7904, 2368
    g = gen(23)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    h = Guarded(tokens, ffn)
    with tide.Compute() as c:
        c.set_test_stall(1_000_000)
        c.gated_forward(tokens, hidden, ffn, x, wg, wu, h)
        with pytest.raises(tide.TideError) as e:
            c.check_device()
        assert e.value.status == tide.TIDE_ERR_TIMEOUT
        c.set_test_stall(0)
        c.gated_forward(tokens, hidden, ffn, x, wg, wu, h)
        c.check_device()
        close(h.view, ref.gated_forward(x, wg, wu, "silu")[0], ref.gated_forward_bound(x, wg, wu, "silu")[0])
        assert h.intact()


@pytest.mark.parametrize("pad_x,pad_h", [(8, 16), (1, 0), (0, 3)])
@pytest.mark.parametrize("tokens", [1, 40, 200])
def test_gated_forward_strided(compute, pad_x, pad_h, tokens):
    hidden, ffn = 264, 392
    g = gen(tokens + pad_x)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    h = Guarded(tokens, ffn, ffn + pad_h)
    compute.gated_forward(tokens, hidden, ffn, strided(x, hidden + pad_x), wg, wu, h, ld_x=hidden + pad_x, ld_h=ffn + pad_h)
    close(h.view, ref.gated_forward(x, wg, wu, "silu")[0], ref.gated_forward_bound(x, wg, wu, "silu")[0])
    assert h.intact()


def run_backward(compute, tokens, hidden, ffn, kind, dh, x, wg, wu, ck=None, h=None, pad=0, **kw):
    dx, dwg, dwu = Guarded(tokens, hidden, hidden + pad), Guarded(ffn, hidden), Guarded(ffn, hidden)
    ws = torch.full((tide.gated_workspace_bytes(tokens, hidden, ffn) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, dwg, dwu, ws, activation=kind, checkpoint=ck, h=h,
                           workspace_bytes=ws.numel() - 256, ld_dx=hidden + pad, **kw)
    assert dx.intact() and dwg.intact() and dwu.intact()
    assert (ws[-256:] == 0xFF).all()
    return dx.view, dwg.view, dwu.view


@pytest.mark.parametrize("tokens,hidden,ffn", GATED_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("with_h", [False, True])
def test_gated_backward_recomputed(compute, tokens, hidden, ffn, kind, with_h):
    g = gen(tokens + hidden + ffn + 1)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    h = Guarded(tokens, ffn) if with_h else None
    got = run_backward(compute, tokens, hidden, ffn, kind, dh, x, wg, wu, h=h)
    want_h, gg, uu = ref.gated_forward(x, wg, wu, kind)
    bh, eg, eu = ref.gated_forward_bound(x, wg, wu, kind)
    want = ref.gated_backward_from(dh, gg, uu, x, wg, wu, kind)
    for a, b, e in zip(got, want, ref.gated_backward_bound(dh, gg, uu, x, wg, wu, kind, eg, eu)):
        close(a, b, e)
    if with_h:
        close(h.view, want_h, bh)
        assert h.intact()


@pytest.mark.parametrize("tokens,hidden,ffn", GATED_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("x8", [False, True])
def test_gated_backward_from_checkpoint(compute, tokens, hidden, ffn, kind, x8):
    g = gen(tokens + hidden + ffn + 2)
    (wg, wu), dh = weights(g, hidden, ffn), randn(g, tokens, ffn)
    x = randn(g, tokens, hidden)
    g8, gs = ref.blocks_store(torch.randn(tokens, ffn, generator=g, device="cuda") * 3, 1)
    u8, us = ref.blocks_store(torch.randn(tokens, ffn, generator=g, device="cuda"), 1)
    xs = ref.blocks_store(x.float(), 1) if x8 else (None, None)
    h = Guarded(tokens, ffn)
    got = run_backward(compute, tokens, hidden, ffn, kind, dh, None if x8 else x, wg, wu,
                       tide.GatedCheckpoint(g8, gs, u8, us, *xs), h=h)
    xv = ref.blocks_value(*xs, 1) if x8 else x.double()
    gg, uu = ref.blocks_value(g8, gs, 1), ref.blocks_value(u8, us, 1)
    want = ref.gated_backward_from(dh, gg, uu, xv, wg, wu, kind)
    for a, b, e in zip(got, want, ref.gated_backward_bound(dh, gg, uu, xv, wg, wu, kind)):
        close(a, b, e)
    arith = ref.arithmetic(gg, kind)
    close(h.view, want[3], want[3].abs() * (arith + ref.U_BF16 * (1 + arith)) + uu.abs() * ref.flushed(gg) + ref.TINY)
    assert h.intact()


@pytest.mark.parametrize("pad", [8, 3])
def test_gated_backward_strided_and_partial(compute, pad):
    tokens, hidden, ffn = 130, 136, 264
    g = gen(pad)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    _, gg, uu = ref.gated_forward(x, wg, wu, "silu")
    _, eg, eu = ref.gated_forward_bound(x, wg, wu, "silu")
    want = ref.gated_backward_from(dh, gg, uu, x, wg, wu, "silu")
    bounds = ref.gated_backward_bound(dh, gg, uu, x, wg, wu, "silu", eg, eu)
    got = run_backward(compute, tokens, hidden, ffn, "silu", strided(dh, ffn + pad), strided(x, hidden + pad), wg, wu,
                       pad=pad, ld_dh=ffn + pad, ld_x=hidden + pad)
    for a, b, e in zip(got, want, bounds):
        close(a, b, e)
    ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu = Guarded(tokens, hidden), Guarded(ffn, hidden), Guarded(ffn, hidden)
    compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, None, None, ws)
    close(dx.view, want[0], bounds[0])
    compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, None, dwg, dwu, ws)
    close(dwg.view, want[1], bounds[1])
    close(dwu.view, want[2], bounds[2])


def test_no_tokens_give_zero_gradients(compute):
    hidden, ffn = 64, 128
    wg = wu = torch.zeros(ffn, hidden, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = Guarded(ffn, hidden), Guarded(ffn, hidden)
    compute.gated_backward(0, hidden, ffn, 0, 0, wg, wu, 0, dwg, dwu, 0, workspace_bytes=0)
    assert (dwg.view == 0).all() and (dwu.view == 0).all() and dwg.intact() and dwu.intact()


def test_sums_of_nothing(compute):
    """No hidden features: h and the gradients of the pre-activations are those
    of zeros.  No ffn features: dx is zero."""
    tokens, ffn = 5, 136
    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, 0, ffn, False)
    compute.gated_forward(tokens, 0, ffn, 0, 0, 0, h, checkpoint=ck)
    assert (h.view == 0).all() and h.intact() and all(b.intact() for b in bufs.values())
    assert (bufs["g8"].view.float() == 0).all() and (bufs["us"].view == 1).all()
    dh = randn(gen(1), tokens, ffn)
    ws = torch.empty(tide.gated_workspace_bytes(tokens, 0, ffn), dtype=torch.uint8, device="cuda")
    h.t.fill_(1.0)
    compute.gated_backward(tokens, 0, ffn, dh, 0, 0, 0, None, None, None, ws, h=h)
    assert (h.view == 0).all() and h.intact()
    hidden = 40
    dx = Guarded(tokens, hidden, 48)
    ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, 0), dtype=torch.uint8, device="cuda")
    x = randn(gen(2), tokens, hidden)
    compute.gated_backward(tokens, hidden, 0, 0, x, 0, 0, dx, None, None, ws, ld_dx=48)
    assert (dx.view == 0).all() and dx.intact()
    x8, xs = Guarded(tokens, hidden, dtype=torch.float8_e4m3fn), Guarded(tokens, 1, dtype=torch.float32)
    compute.gated_forward(tokens, hidden, 0, x, 0, 0, 0, checkpoint=tide.GatedCheckpoint(0, 0, 0, 0, x8, xs))
    codes, scales = ref.blocks_store(x.float().cpu(), 1)
    assert torch.equal(xs.view.cpu(), scales) and x8.intact() and xs.intact()
    same_codes(x8.view.cpu(), codes)


def test_nan_and_infinity_stay_in_their_token(compute):
    """A token that holds NaN or infinities spoils its own row of h only, and
    its checkpoint shows them as NaN."""
    tokens, hidden, ffn = 150, 256, 264
    g = gen(9)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    clean = Guarded(tokens, ffn)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, clean)
    x[3, 7], x[140, 255] = math.nan, math.inf
    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, hidden, ffn, True)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck)
    rows = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rows[[3, 140]] = False
    assert torch.equal(h.view[rows], clean.view[rows])
    assert torch.isnan(h.view[3]).all() and not torch.isfinite(h.view[140]).any()
    for n in ("g8", "u8"):
        bad = torch.isnan(bufs[n].view.float())
        assert not bad[rows].any() and bad[3].all() and bad[140].all()
    assert torch.equal(torch.isnan(bufs["x8"].view.float()), ~torch.isfinite(x))


@pytest.mark.parametrize("value", [0.0, 30.0, 90.0, 1e4, 1e18])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_saturated_gates(compute, value, kind):
    """Gates far out on both sides keep their limits, forward and backward."""
    tokens, hidden, ffn = 5, 8, 128
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 1.0
    wg = torch.zeros(ffn, hidden, dtype=torch.bfloat16, device="cuda")
    wg[::2, 0], wg[1::2, 0] = value, -value
    wu = torch.zeros_like(wg)
    wu[:, 1] = 0.5
    dh = torch.ones(tokens, ffn, dtype=torch.bfloat16, device="cuda")
    h = Guarded(tokens, ffn)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, activation=kind)
    want, gg, uu = ref.gated_forward(x, wg, wu, kind)
    close(h.view, want, ref.gated_forward_bound(x, wg, wu, kind)[0])
    got = run_backward(compute, tokens, hidden, ffn, kind, dh, x, wg, wu)
    bounds = ref.gated_backward_bound(dh, gg, uu, x, wg, wu, kind)
    for a, b, e in zip(got, ref.gated_backward_from(dh, gg, uu, x, wg, wu, kind), bounds):
        close(a, b, e)


# merged dX and dW; dX beside dW; sums in parts; 256-row tiles throughout
@pytest.mark.parametrize("tokens,hidden,ffn", [(64, 256, 704), (40, 264, 2056), (700, 264, 2056), (300, 136, 2568)])
def test_streams_and_capture(compute, tokens, hidden, ffn):
    """Calls follow their own stream, and replay from a CUDA graph."""
    g = gen(4)
    (wg, wu), dh = weights(g, hidden, ffn), randn(g, tokens, ffn)
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    h, dx, dwg, dwu = (torch.empty(*s, dtype=torch.bfloat16, device="cuda")
                       for s in ((tokens, ffn), (tokens, hidden), (ffn, hidden), (ffn, hidden)))
    ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    def step():
        compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, stream=torch.cuda.current_stream())
        compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, dwg, dwu, ws, stream=torch.cuda.current_stream())

    def check():
        want, gg, uu = ref.gated_forward(x, wg, wu, "silu")
        bh, eg, eu = ref.gated_forward_bound(x, wg, wu, "silu")
        close(h, want, bh)
        for a, b, e in zip((dx, dwg, dwu), ref.gated_backward_from(dh, gg, uu, x, wg, wu, "silu"),
                           ref.gated_backward_bound(dh, gg, uu, x, wg, wu, "silu", eg, eu)):
            close(a, b, e)

    with torch.cuda.stream(s):
        x.copy_(randn(gen(7), tokens, hidden))
        step()
    s.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (11, 12):
        x.copy_(randn(gen(seed), tokens, hidden))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check()


def test_streams_side_by_side(compute):
    """Calls of every kind on three streams at once, one handle, give what they
    give one after the other."""
    g = gen(55)

    class Job:
        def __init__(self, tokens, hidden, ffn):
            self.size = tokens, hidden, ffn
            self.x, self.dh, (self.wg, self.wu) = randn(g, tokens, hidden), randn(g, tokens, ffn), weights(g, hidden, ffn)
            (self.a, self.sa), (self.b, self.sb) = fp8(g, tokens, ffn, 1), fp8(g, hidden, ffn, 128)
            new = dict(device="cuda", dtype=torch.bfloat16)
            self.out = [torch.empty(*s, **new) for s in
                        ((tokens, ffn), (tokens, hidden), (ffn, hidden), (ffn, hidden), (tokens, hidden))]
            self.codes = torch.empty(tokens, ffn, dtype=torch.uint8, device="cuda")
            self.scales = torch.empty(tokens, -(-ffn // 128), device="cuda")
            self.ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")

        def run(self, stream):
            m, k, f = self.size
            h, dx, dwg, dwu, y = self.out
            compute.gated_forward(m, k, f, self.x, self.wg, self.wu, h, stream=stream)
            compute.fp8_matmul(m, k, f, self.a, self.sa, self.b, self.sb, y, stream=stream)
            compute.fp8_store(m, f, h, self.codes, self.scales, stream=stream)
            compute.gated_backward(m, k, f, self.dh, self.x, self.wg, self.wu, dx, dwg, dwu, self.ws, stream=stream)

        def results(self):
            return [t.clone() for t in self.out + [self.codes, self.scales]]

    jobs = [Job(*s) for s in ((5, 256, 704), (700, 264, 2056), (40, 512, 2560), (300, 1024, 3328), (130, 2048, 768))]
    torch.cuda.synchronize()
    want = []
    for j in jobs:
        j.run(None)
        torch.cuda.synchronize()
        want.append(j.results())
        for t in j.out:
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(20):
        for i, j in enumerate(jobs):
            j.run(streams[(i + turn) % 3] if turn == 0 else streams[i % 3])
        if turn == 0:
            torch.cuda.synchronize()  # jobs change streams after this turn
    torch.cuda.synchronize()
    compute.check_device()
    for j, w in zip(jobs, want):
        for a, b in zip(j.results(), w):
            assert torch.equal(a, b)


def test_first_call_is_not_captured():
    with tide.Compute() as c:
        src = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
        codes, scales = torch.empty(4, 128, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(tide.TideError) as e:
                c.fp8_store(4, 128, src, codes, scales, stream=torch.cuda.current_stream())
        assert e.value.status == tide.TIDE_ERR_UNSUPPORTED


def test_same_results_every_time(compute):
    tokens, hidden, ffn = 90, 520, 1032
    g = gen(21)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    first = [t.clone() for t in run_backward(compute, tokens, hidden, ffn, "silu", dh, x, wg, wu)]
    for _ in range(5):
        for a, b in zip(first, run_backward(compute, tokens, hidden, ffn, "silu", dh, x, wg, wu)):
            assert torch.equal(a, b)


def test_wait_that_runs_out_is_reported():
    tokens, hidden, ffn = 300, 256, 704
    g = gen(30)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    h = Guarded(tokens, ffn)
    (a, sa), (b, sb) = fp8(g, 2000, hidden, 1), fp8(g, 5000, hidden, 128)
    out = Guarded(2000, 5000)
    with tide.Compute() as c:
        c.check_device()
        c.set_test_stall(1_000_000)
        for call in (lambda: c.gated_forward(tokens, hidden, ffn, x, wg, wu, h),
                     lambda: c.gated_forward(2, hidden, ffn, x, wg, wu, h),
                     lambda: c.fp8_matmul(2000, 5000, hidden, a, sa, b, sb, out),
                     lambda: c.fp8_matmul(2000, 5000, hidden, a, sa, b, sb, out, any_scales=True),
                     lambda: c.fp8_matmul(2, 5000, hidden, a, sa, b, sb, out),
                     lambda: run_backward(c, tokens, hidden, ffn, "silu", dh, x, wg, wu)):
            call()
            with pytest.raises(tide.TideError) as e:
                c.check_device()
            assert e.value.status == tide.TIDE_ERR_TIMEOUT
            c.check_device()  # cleared
        c.set_test_stall(0)
        c.gated_forward(tokens, hidden, ffn, x, wg, wu, h)
        c.check_device()
        close(h.view, ref.gated_forward(x, wg, wu, "silu")[0], ref.gated_forward_bound(x, wg, wu, "silu")[0])
        assert h.intact()


def test_feed_forward_unit_learns():
    """The operators together, from the gathered buffer to the shards: the
    example's loss falls step by step, and after one step each shard's update
    is the mean of the ranks' gradients computed in 64 bits."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward_unit.py")
    spec = importlib.util.spec_from_file_location("feed_forward_unit", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=20)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.8 * losses[0]

    unit, acts = m.Unit(3, 136, 264), m.Activations(50, 136, 264)
    g = gen(3)
    xs = [randn(g, 50, 136) for _ in range(3)]
    goals = [torch.randn(50, 136, generator=g, device="cuda") for _ in range(3)]
    with tide.Compute() as c:
        m.step(unit, c, acts, xs, goals, 0.0)
    gate, up, down = (p.double() for p in unit.params)
    mean = [torch.zeros_like(p) for p in (gate, up, down)]
    for x, goal in zip(xs, goals):
        h, gg, uu = ref.gated_forward(x, gate, up, "silu")
        dy = 2 * (h @ down.T - goal.double()) / goal.numel()
        dh = dy @ down
        _, dg, du, _ = ref.gated_backward_from(dh, gg, uu, x, gate, up, "silu")
        for acc, v in zip(mean, (dg, du, dy.T @ h)):
            acc += v / 3
    for p, want in enumerate(mean):
        rows = unit.shapes[p][0]
        got = torch.cat([unit.updates[r][p] for r in range(3)])[:rows].double()
        # e4m3 rounds each of g, u, x, h and the down weights by up to 2^-4:
        # as independent errors (rms 2^-5.6 each) well under a fifth in norm
        assert float((got - want).norm() / want.norm()) < 0.2


# ------------------------------------------------- offsets past 32 bits

def pick8(codes, rows):
    return codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn)


@pytest.mark.parametrize("rows", [70001, 100003])  # past 2^31 elements; past 3 * 2^30
@pytest.mark.parametrize("cols", [32776, 32777])
def test_blocks_past_32_bits(compute, rows, cols):
    src = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = gen(rows + cols)
    picks = [0, 2 ** 31 // cols // 128 * 128, rows // 128 * 128 - 128]
    src.zero_()
    for r in picks:
        src[r:r + 128] = randn(g, 128, cols)
    for block_rows in (1, 128):
        codes = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(-(-rows // block_rows), -(-cols // 128), device="cuda")
        back = torch.empty_like(src)
        compute.fp8_store(rows, cols, src, codes, scales, block_rows=block_rows)
        compute.fp8_restore(rows, cols, codes, scales, back, block_rows=block_rows)
        for r in picks:
            v = src[r:r + 128].float()
            j = torch.arange(cols, device="cuda") // 128
            top = torch.zeros(128 // block_rows, scales.shape[1], device="cuda")
            i = torch.arange(128, device="cuda") // block_rows
            top = top.reshape(-1).scatter_reduce(0, (i[:, None] * scales.shape[1] + j).reshape(-1), v.abs().reshape(-1),
                                                 "amax").view_as(top)
            s = scales[r // block_rows:(r + 128) // block_rows]
            assert ((top <= 448 * s) & (top > 224 * s)).all()
            each = s[i][:, j]
            assert torch.equal(codes[r:r + 128].float(), (v / each).to(torch.float8_e4m3fn).float())
            assert torch.equal(back[r:r + 128].float(), codes[r:r + 128].float() * each)
        assert float(back.abs().float().sum(dtype=torch.float64)) == sum(
            float(back[r:r + 128].abs().float().sum(dtype=torch.float64)) for r in picks)
        del codes, scales, back


def test_gated_past_32_bits(compute):
    tokens, hidden, ffn = 80003, 64, 28680
    g = gen(99)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    dh = randn(g, tokens, ffn)
    new = dict(device="cuda", dtype=torch.bfloat16)
    h, dx = torch.empty(tokens, ffn, **new), torch.empty(tokens, hidden, **new)
    dwg, dwu = torch.empty(ffn, hidden, **new), torch.empty(ffn, hidden, **new)
    codes = [torch.empty(tokens, ffn, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.empty(tokens, -(-ffn // 128), device="cuda") for _ in range(2)]
    ck = tide.GatedCheckpoint(codes[0], scales[0], codes[1], scales[1])
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck)
    ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
    rows = torch.tensor([0, 40000, 2 ** 31 // ffn, 2 ** 31 // ffn + 1, 79999, tokens - 1], device="cuda")
    cols = torch.tensor([0, 1, 14340, ffn - 129, ffn - 1], device="cuda")
    want, gg, uu = ref.gated_forward(x[rows], wg, wu, "silu")
    bh, eg, eu = ref.gated_forward_bound(x[rows], wg, wu, "silu")
    close(h[rows], want, bh)
    close_to_stored(pick8(codes[0], rows), scales[0][rows], gg, eg)
    close_to_stored(pick8(codes[1], rows), scales[1][rows], uu, eu)
    for kept in (None, ck):
        h.fill_(0)
        compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, dwg, dwu, ws, checkpoint=kept, h=h)
        compute.check_device()
        if kept is None:
            pre = ref.gated_forward(x[rows], wg, wu, "silu")[1:]
            err = ref.gated_forward_bound(x[rows], wg, wu, "silu")[1:]
            part = ref.gated_forward(x, wg[cols], wu[cols], "silu")[1:]
            part_err = ref.gated_forward_bound(x, wg[cols], wu[cols], "silu")[1:]
        else:
            pre = [ref.blocks_value(pick8(codes[i], rows), scales[i][rows], 1) for i in range(2)]
            j = cols // 128
            part = [codes[i].view(torch.uint8)[:, cols].view(torch.float8_e4m3fn).float().double() * scales[i][:, j].double() for i in range(2)]
            err = part_err = (0.0, 0.0)
        want = ref.gated_backward_from(dh[rows], *pre, x[rows], wg, wu, "silu")
        close(dx[rows], want[0], ref.gated_backward_bound(dh[rows], *pre, x[rows], wg, wu, "silu", *err)[0])
        want = ref.gated_backward_from(dh[:, cols], *part, x, wg[cols], wu[cols], "silu")
        bounds = ref.gated_backward_bound(dh[:, cols], *part, x, wg[cols], wu[cols], "silu", *part_err)
        close(dwg[cols], want[1], bounds[1])
        close(dwu[cols], want[2], bounds[2])
        hw = ref.act(pre[0], "silu") * pre[1]
        off = bh if kept is None else hw.abs() * (ref.arithmetic(pre[0], "silu") + 1.01 * ref.U_BF16) + ref.TINY * (
            1 + pre[1].abs() * (1 + pre[0].abs()) ** 3)
        close(h[rows], hw, off)


@pytest.mark.parametrize("any_scales", [False, True])
def test_matmul_past_32_bits(compute, any_scales):
    m, n, k = 80003, 28680, 144
    g = gen(98)
    (a, sa), (b, sb) = fp8(g, m, k, 1, any_scales), fp8(g, n, k, 128, any_scales)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out, any_scales=any_scales)
    rows = torch.tensor([0, 2 ** 31 // n, 2 ** 31 // n + 1, m - 1], device="cuda")
    close(out[rows], *ref.matmul(pick8(a, rows), sa[rows], b, sb))


# ------------------------------------- one warp's wait runs out, others' do not

def late_calls():
    """(name, call(compute), results) of every tensor-core kernel: one tile a
    pair of CTAs and several, whole contractions and split ones."""
    g = gen(60)
    calls = []

    def matmul(m, n, k, any_scales=False):
        (a, sa), (b, sb) = fp8(g, m, k, 1), fp8(g, n, k, 128)
        out = Guarded(m, n)
        calls.append((f"matmul {m} {n} {k} {any_scales}",
                      lambda c: c.fp8_matmul(m, n, k, a, sa, b, sb, out, any_scales=any_scales), [out]))

    def gated(tokens, hidden, ffn):
        x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
        h, dx = Guarded(tokens, ffn), Guarded(tokens, hidden)
        dwg, dwu = Guarded(ffn, hidden), Guarded(ffn, hidden)
        ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
        calls.append((f"forward {tokens} {hidden} {ffn}",
                      lambda c: c.gated_forward(tokens, hidden, ffn, x, wg, wu, h), [h]))
        calls.append((f"backward {tokens} {hidden} {ffn}",
                      lambda c: c.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, dwg, dwu, ws), [dx, dwg, dwu]))

    matmul(2, 264, 2064)
    matmul(64, 136, 8192)
    matmul(300, 5200, 400)
    matmul(2100, 5200, 1040)
    matmul(300, 5200, 400, True)
    matmul(2100, 5200, 1040, True)
    matmul(1014, 752, 9200)
    gated(2, 256, 704)
    gated(64, 512, 2560)
    gated(3000, 72, 136)
    gated(4200, 264, 2056)
    gated(200, 7904, 2368)
    return calls


def test_warp_whose_wait_runs_out_leaves_alone():
    """One warp of a kernel gives up while the sums are there: the call ends, the
    error is reported, nothing outside the outputs is written, and the same call
    afterwards gives what it gave before."""
    with tide.Compute() as c:
        for name, call, results in late_calls():
            call(c)
            c.check_device()
            want = [r.view.clone() for r in results]
            c.set_test_late_warp(1_000_000)
            for _ in range(3):
                call(c)
                with pytest.raises(tide.TideError) as e:
                    c.check_device()
                assert e.value.status == tide.TIDE_ERR_TIMEOUT, name
                assert all(r.intact() for r in results), name
            c.set_test_late_warp(0)
            call(c)
            c.check_device()
            for r, w in zip(results, want):
                assert torch.equal(r.view, w), name


@pytest.mark.parametrize("tokens,hidden,ffn", [(3000, 72, 136), (4200, 264, 2056), (300, 1544, 2600)])
def test_half_a_block_s_warp_that_leaves_takes_the_other_along(tokens, hidden, ffn):
    """A checkpoint's block is two warps' and they meet over its maximum: where
    one gives up the other does not wait for it."""
    g = gen(61)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, hidden, ffn, False)
    with tide.Compute() as c:
        c.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck)
        c.check_device()
        want = [b.view.clone().view(torch.uint8) for b in [h, *bufs.values()]]
        c.set_test_late_warp(1_000_000)
        for _ in range(3):
            c.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck)
            with pytest.raises(tide.TideError) as e:
                c.check_device()
            assert e.value.status == tide.TIDE_ERR_TIMEOUT
            assert h.intact() and all(b.intact() for b in bufs.values())
        c.set_test_late_warp(0)
        c.gated_forward(tokens, hidden, ffn, x, wg, wu, h, checkpoint=ck)
        c.check_device()
        for b, w in zip([h, *bufs.values()], want):
            assert torch.equal(b.view.view(torch.uint8), w)


# ------------------------- more columns than 65535 tiles of the plain kernels

@pytest.mark.parametrize("tokens,hidden,ffn", [(1, 1, 9_000_001), (2, 3, 8_388_481), (1, 9_000_001, 1), (2, 8_388_481, 3)])
def test_gated_very_wide(compute, tokens, hidden, ffn):
    g = gen(tokens + hidden + ffn)
    x, (wg, wu), dh = randn(g, tokens, hidden), weights(g, hidden, ffn), randn(g, tokens, ffn)
    h = Guarded(tokens, ffn)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h)
    want, gg, uu = ref.gated_forward(x, wg, wu, "silu")
    bh, eg, eu = ref.gated_forward_bound(x, wg, wu, "silu")
    close(h.view, want, bh)
    assert h.intact()
    got = run_backward(compute, tokens, hidden, ffn, "silu", dh, x, wg, wu)
    for a, b, e in zip(got, ref.gated_backward_from(dh, gg, uu, x, wg, wu, "silu"),
                       ref.gated_backward_bound(dh, gg, uu, x, wg, wu, "silu", eg, eu)):
        close(a, b, e)


@pytest.mark.parametrize("m,n,k", [(1, 9_000_001, 16), (3, 8_388_481, 5)])
@pytest.mark.parametrize("any_scales", [False, True])
def test_matmul_very_wide(compute, m, n, k, any_scales):
    g = gen(m + n + k)
    (a, sa), (b, sb) = fp8(g, m, k, 1, any_scales), fp8(g, n, k, 128, any_scales)
    out = Guarded(m, n)
    compute.fp8_matmul(m, n, k, a, sa, b, sb, out, any_scales=any_scales)
    close(out.view, *ref.matmul(a, sa, b, sb))
    assert out.intact()


# ------------------------------- two scales whose product fp32 does not hold

# few tokens; unaligned; 256-row tiles; clusters of them
WIDE_SCALE_SHAPES = [(4, 264, 1024), (40, 264, 1024), (7, 130, 1027), (300, 5200, 1024), (1014, 752, 9216)]


@pytest.mark.parametrize("m,n,k", WIDE_SCALE_SHAPES)
@pytest.mark.parametrize("sa,sb,any_scales", [(2.0 ** 70, 2.0 ** 60, False), (2.0 ** 70, 2.0 ** 60, True), (2.0 ** 127, 2.0 ** 127, False),
                                              (2.0 ** 127, 2.0 ** 127, True), (-1.5 * 2.0 ** 70, 1.25 * 2.0 ** 60, True)])
def test_matmul_scales_whose_product_is_past_fp32(compute, m, n, k, sa, sb, any_scales):
    """A sum of zeros is zero whatever its scales; one small product is finite
    where the value is; what is past fp32 is infinite.  Other blocks of the row
    are as they were."""
    one = torch.ones(m, n, dtype=torch.float64, device="cuda")
    a = torch.zeros(m, k, device="cuda").to(torch.float8_e4m3fn)
    b = torch.zeros(n, k, device="cuda").to(torch.float8_e4m3fn)
    nb = -(-k // 128)
    za, zb = torch.full((m, nb), sa, device="cuda"), torch.full((-(-n // 128), nb), sb, device="cuda")
    za[:, 1], zb[:, 1] = 1.0, 0.5
    bv = b.view(torch.uint8)
    av = a.view(torch.uint8)
    bv[:, 128], av[:, 128] = 0x38, 0x40  # 1 and 2: the second block's sum is 2, its value 1
    out = Guarded(m, n)
    compute.fp8_matmul(m, n, k, a, za, b, zb, out, any_scales=any_scales)
    close(out.view, one, 0.0 * one)
    if abs(sa * sb) < 2.0 ** 140:
        av[1, 5], bv[:, 5] = 0x01, 0x01  # 2^-18 in all
        compute.fp8_matmul(m, n, k, a, za, b, zb, out, any_scales=any_scales)
        want = one.clone()
        want[1] += 2.0 ** -18 * sa * sb
        close(out.view, want, want.abs() * ref.U_BF16)
    av[2, 7], bv[:, 7] = 0x7E, 0x7E
    compute.fp8_matmul(m, n, k, a, za, b, zb, out, any_scales=any_scales)
    assert (out.view[2] == math.copysign(math.inf, sa)).all()
    assert torch.isfinite(out.view[0]).all() and torch.isfinite(out.view[3:]).all() and out.intact()


@pytest.mark.parametrize("m,n,k", WIDE_SCALE_SHAPES)
@pytest.mark.parametrize("sa,sb,any_scales", [(2.0 ** -80, 2.0 ** -72, False), (2.0 ** -80, 2.0 ** -72, True),
                                              (2.0 ** -126, 2.0 ** -26, False), (1.5 * 2.0 ** -80, 1.25 * 2.0 ** -72, True),
                                              (1e-42, 2.0 ** -12, True)])
def test_matmul_scales_whose_product_is_below_fp32(compute, m, n, k, sa, sb, any_scales):
    """Block sums times such scales add up to what fp32 holds.  Every term is
    up to 2^-126, of which fp32 keeps at least 2^-149: within 2^-149 for each
    block, its sum's and the scales' own rounding beside it."""
    a = torch.full((m, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    b = torch.full((n, k), 416.0, device="cuda").to(torch.float8_e4m3fn)
    nb = -(-k // 128)
    za, zb = torch.full((m, nb), sa, device="cuda"), torch.full((-(-n // 128), nb), sb, device="cuda")
    out = Guarded(m, n)
    compute.fp8_matmul(m, n, k, a, za, b, zb, out, any_scales=any_scales)
    want = ref.blocks_value(a, za, 1) @ ref.blocks_value(b, zb, 128).T
    assert float(want.min()) > 2.0 ** -126
    off = want * (k + 8) * ref.U_F32 + nb * 2.0 ** -149
    close(out.view, want, off + ref.U_BF16 * (want + off))
    assert out.intact()


# ------------------------------------------------- gates far below zero

FAR_SHAPES = [(1, 8, 136), (40, 264, 392), (3, 9, 131), (3000, 72, 136)]  # few tokens, plain kernels, 256-row tiles


@pytest.mark.parametrize("tokens,hidden,ffn", FAR_SHAPES)
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_far_below_zero(compute, tokens, hidden, ffn, kept, kind):
    """The activations fall to 1e-37 and on into the subnormal numbers: what
    fp32 holds of the sigmoid is there in h, dU and dG.  Rounding as
    ref.arithmetic has it, two units of the smallest subnormal number times
    what the sigmoid is multiplied by, bf16's rounding last."""
    if kept:  # as e4m3 has them
        values = [-80.0, -88.0, -96.0] if kind == "silu" else [-9.0, -10.0, -11.0]
    elif kind == "silu":
        values = [-80.0, -84.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -92.0, -94.0, -96.0]
    else:
        values = [-9.5, -9.875, -10.0, -10.0625, -10.125, -10.1875, -10.25, -10.375, -10.5, -10.625]
    values = torch.tensor(values, device="cuda")
    g = values[torch.arange(ffn, device="cuda") % len(values)]
    up = 2.0 ** 90
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, :2] = 1.0
    wg, wu = (torch.zeros(ffn, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 1] = g.bfloat16(), up
    dh = torch.ones(tokens, ffn, dtype=torch.bfloat16, device="cuda")
    gd = g.double()
    a, d = ref.act(gd, kind), ref.act_grad(gd, kind)
    rel = ref.arithmetic(gd, kind)
    slope = 1.0 if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * gd ** 2)
    off_a, off_d = gd.abs() * 2.0 ** -148, (1 + gd.abs() * slope) * 2.0 ** -148
    tiny = 2.0 ** -134  # half of bf16's smallest subnormal number

    def rounded(v, e):
        return e + ref.U_BF16 * (v.abs() + e) + tiny

    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, hidden, ffn, False) if kept else ({}, None)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, activation=kind, checkpoint=ck)
    one = torch.ones(tokens, 1, dtype=torch.float64, device="cuda")
    want_h, bound_h = one * (a * up), one * rounded(a * up, (a.abs() * rel + off_a) * up)
    close(h.view, want_h, bound_h)
    h.t.zero_()
    _, dwg, dwu = run_backward(compute, tokens, hidden, ffn, kind, dh, x, wg, wu, ck, h=h)
    close(h.view, want_h, bound_h)
    sums = tokens * (tokens + 8) * ref.U_F32
    for got, v, scale, off in ((dwg, d, up, off_d), (dwu, a, 1.0, off_a)):
        e = rounded(v * scale, (v.abs() * 2 * rel + off) * scale)  # dG or dU
        want = tokens * v * scale
        close(got[:, 0], want, rounded(want, tokens * e + sums * (v.abs() * scale + e)))


@pytest.mark.parametrize("tokens,hidden,ffn", FAR_SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("kept", [False, True])
def test_gates_near_the_largest_number(compute, tokens, hidden, ffn, kind, kept):
    """Twice the gate is past fp32, the slope 1 or 0 is not: everything here is
    a power of two or exact in bf16, so every result is."""
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** 64, 1.0
    wg, wu = (torch.zeros(ffn, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[::2, 0], wg[1::2, 0], wu[:, 1] = 1.75 * 2.0 ** 63, -1.75 * 2.0 ** 63, 1.0
    dh = torch.zeros(tokens, ffn, dtype=torch.bfloat16, device="cuda")
    dh[0] = 2.0 ** -70
    h = Guarded(tokens, ffn)
    bufs, ck = checkpoint(tokens, hidden, ffn, False) if kept else ({}, None)
    compute.gated_forward(tokens, hidden, ffn, x, wg, wu, h, activation=kind, checkpoint=ck)
    on = (torch.arange(ffn, device="cuda") % 2 == 0).double()
    g = 1.75 * 2.0 ** 127
    assert torch.equal(h.view.double(), (on * g).expand(tokens, ffn))
    _, dwg, dwu = run_backward(compute, tokens, hidden, ffn, kind, dh, x, wg, wu, ck)
    assert torch.equal(dwg[:, 1].double(), on * 2.0 ** -70)
    assert torch.equal(dwg[:, 0].double(), on * 2.0 ** -6)
    assert torch.equal(dwu[:, 1].double(), on * g * 2.0 ** -70)


# by the few-token kernel; joined from parts; in one launch with dW
@pytest.mark.parametrize("tokens,hidden,ffn", [(4, 1032, 14336), (64, 512, 2048), (250, 256, 704)])
def test_dx_follows_its_gradients(compute, tokens, hidden, ffn):
    """dX beside dW reads the gradients of its own call: calls back to back, on a
    stream and from a graph, give what dX alone gives, whatever came before."""
    g = gen(tokens)
    x, (wg, wu) = randn(g, tokens, hidden), weights(g, hidden, ffn)
    dhs = [randn(gen(i), tokens, ffn) for i in range(8)]
    ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
    alone, both = ([torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda") for _ in dhs] for _ in range(2))
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)

    def run(dxs, with_w):
        for dh, dx in zip(dhs, dxs):
            compute.gated_backward(tokens, hidden, ffn, dh, x, wg, wu, dx, dwg if with_w else None, dwu if with_w else None,
                                   ws, stream=torch.cuda.current_stream())

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run(alone, False)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(both, True)
    for turn in range(20):
        if turn % 2:
            graph.replay()
        else:
            with torch.cuda.stream(s):
                run(both, True)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a, b)
            b.zero_()
        torch.cuda.synchronize()


class Mixed:
    """Calls of every kind on one set of buffers."""

    def __init__(self, g, tokens, hidden, ffn):
        self.size = tokens, hidden, ffn
        self.x, self.dh, (self.wg, self.wu) = randn(g, tokens, hidden), randn(g, tokens, ffn), weights(g, hidden, ffn)
        (self.a, self.sa), (self.b, self.sb) = fp8(g, tokens, ffn, 1), fp8(g, hidden, ffn, 128)
        new = dict(device="cuda", dtype=torch.bfloat16)
        self.out = [torch.empty(*s, **new) for s in
                    ((tokens, ffn), (tokens, hidden), (ffn, hidden), (ffn, hidden), (tokens, hidden), (tokens, ffn))]
        self.codes, self.scales = (torch.empty(2 * tokens, ffn, dtype=torch.uint8, device="cuda"),
                                   torch.empty(2 * tokens, -(-ffn // 128), device="cuda"))
        self.ck = tide.GatedCheckpoint(self.codes[:tokens], self.scales[:tokens], self.codes[tokens:], self.scales[tokens:]) \
            if tokens * ffn % 16 == 0 else None
        self.ws = torch.empty(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8, device="cuda")

    def run(self, c, stream):
        m, k, f = self.size
        h, dx, dwg, dwu, y, back = self.out
        c.gated_forward(m, k, f, self.x, self.wg, self.wu, h, checkpoint=self.ck, stream=stream)
        c.fp8_matmul(m, k, f, self.a, self.sa, self.b, self.sb, y, stream=stream)
        c.gated_backward(m, k, f, self.dh, self.x, self.wg, self.wu, dx, dwg, dwu, self.ws, checkpoint=self.ck, stream=stream)
        if self.ck:
            c.fp8_restore(m, f, self.codes, self.scales, back, stream=stream)
        else:
            back.zero_()

    def results(self):
        return [t.clone() for t in self.out]


def test_jobs_change_streams(compute):
    """One handle, workspace and set of buffers on another stream each turn,
    in order by events: every turn gives the same, from cleared outputs."""
    g = gen(56)
    jobs = [Mixed(g, *s) for s in ((16, 256, 704), (700, 264, 2056), (40, 512, 2560), (304, 1024, 3328), (128, 2048, 768))]
    torch.cuda.synchronize()
    want = []
    for j in jobs:
        j.run(compute, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(j.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    last, got = [None] * len(jobs), [[] for _ in jobs]
    for turn in range(6):
        for i, j in enumerate(jobs):
            with torch.cuda.stream(streams[(i + turn) % 3]):
                if last[i]:
                    last[i].wait()
                for t in j.out:
                    t.zero_()
                j.run(compute, torch.cuda.current_stream())
                got[i].append(j.results())
                last[i] = torch.cuda.Event()
                last[i].record()
    torch.cuda.synchronize()
    compute.check_device()
    for turns, w in zip(got, want):
        for results in turns:
            for a, b in zip(results, w):
                assert torch.equal(a, b)


def test_captured_fork_and_join(compute):
    """Calls captured on two streams that part and meet again: the calls behind
    the meeting have the ends of both ahead of them."""
    g = gen(57)
    one, two, both = (Mixed(g, *s) for s in ((128, 512, 2560), (304, 1024, 768), (64, 256, 704)))
    k, f = both.size[1:]
    seen = torch.empty(64, f, dtype=torch.bfloat16, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        compute.gated_forward(64, k, f, both.x, both.wg, both.wu, both.out[0], stream=s1)
        fork.record(s1)
        s2.wait_event(fork)
        with torch.cuda.stream(s1):
            one.run(compute, s1)
        with torch.cuda.stream(s2):
            two.run(compute, s2)
            # what the call behind the meeting reads comes from this side
            compute.fp8_restore(64, f, two.codes, two.scales, seen, stream=s2)
        join.record(s2)
        s1.wait_event(join)
        compute.gated_backward(64, k, f, seen, both.x, both.wg, both.wu, both.out[1], both.out[2], both.out[3], both.ws, stream=s1)

    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    want = [j.results() for j in (one, two, both)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        step()
    for _ in range(10):
        for j in (one, two, both):
            for t in j.out:
                t.zero_()
        seen.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, w in zip((one, two, both), want):
            # both.out[4] and [5] are not written here
            for a, b in list(zip(j.results(), w))[:4 if j is both else 6]:
                assert torch.equal(a, b)
