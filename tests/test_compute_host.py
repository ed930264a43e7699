"""Feed-forward operators without a GPU: refusals, sizes and the formulas the
GPU tests compare with."""
import ctypes

import numpy
import pytest
import torch

import ffn_reference as ref
import layout_aware_collectives_gb300 as tide

A = 4096  # a 16-byte aligned address that refused calls never read


@pytest.fixture
def compute():
    with tide.Compute() as c:
        yield c


def refused(status, fn, *args, **kw):
    with pytest.raises(tide.TideError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)


BAD, MIS = tide.TIDE_ERR_INVALID_ARG, tide.TIDE_ERR_MISALIGNED


def test_store_and_restore_refuse(compute):
    for f in (lambda *a, **k: compute.fp8_store(*a, **k), lambda r, c, s, o, z, **k: compute.fp8_restore(r, c, o, z, s, **k)):
        refused(BAD, f, 4, 128, A, A, A, block_rows=64)
        refused(BAD, f, -1, 128, A, A, A)
        refused(BAD, f, 1 << 31, 1, A, A, A)
        refused(BAD, f, (1 << 31) - 1, (1 << 31) - 1, A, A, A)
        refused(BAD, f, 4, 128, 0, A, A)
        refused(BAD, f, 4, 128, A, 0, A)
        refused(BAD, f, 4, 128, A, A, 0)
        refused(MIS, f, 4, 128, A + 2, A, A)
        refused(MIS, f, 4, 128, A, A + 1, A)
        refused(MIS, f, 4, 128, A, A, A + 2)
        f(0, 128, 0, 0, 0)  # nothing to do, no device touched
        f(4, 0, 0, 0, 0)
    refused(BAD, compute.fp8_store, 4, 128, A, A, A, ld_src=127)
    refused(BAD, compute.fp8_restore, 4, 128, A, A, A, ld_dst=127)


def test_matmul_refuses(compute):
    ok = [4, 8, 128, A, A, A, A, A]
    for i, v, st in ((0, -1, BAD), (1, 1 << 31, BAD), (2, -5, BAD), (3, 0, BAD), (4, 0, BAD), (5, A + 8, MIS),
                     (6, A + 1, MIS), (7, A + 2, MIS), (7, 0, BAD)):
        bad = list(ok)
        bad[i] = v
        refused(st, compute.fp8_matmul, *bad)
    refused(BAD, compute.fp8_matmul, *ok, ld_out=7)
    compute.fp8_matmul(0, 8, 128, 0, 0, A, A, 0)
    compute.fp8_matmul(4, 0, 128, A, A, 0, 0, 0)


def test_forward_refuses(compute):
    ok = [4, 128, 256, A, A, A, A]
    for i, v, st in ((0, -1, BAD), (1, 1 << 31, BAD), (2, -2, BAD), (3, 0, BAD), (3, A + 2, MIS), (4, 0, BAD),
                     (5, A + 8, MIS), (6, 0, BAD)):
        bad = list(ok)
        bad[i] = v
        refused(st, compute.gated_forward, *bad)
    refused(BAD, compute.gated_forward, *ok, ld_x=127)
    refused(BAD, compute.gated_forward, *ok, ld_h=255)
    refused(BAD, compute.gated_forward, *ok, activation=7)
    with pytest.raises(ValueError):
        compute.gated_forward(*ok, activation="swish")
    for i in range(4):
        parts = [A] * 4
        parts[i] = 0
        refused(BAD, compute.gated_forward, *ok, checkpoint=tide.GatedCheckpoint(*parts))
    refused(BAD, compute.gated_forward, *ok, checkpoint=tide.GatedCheckpoint(A, A, A, A, A, 0))
    refused(MIS, compute.gated_forward, *ok, checkpoint=tide.GatedCheckpoint(A, A, A + 8, A))
    compute.gated_forward(0, 128, 256, 0, A, A, 0)


def test_backward_refuses(compute):
    n = tide.gated_workspace_bytes(4, 128, 256)
    ok = [4, 128, 256, A, A, A, A, A, A, A, A]
    kw = dict(workspace_bytes=n)
    for i, v, st in ((0, -1, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (6, A + 2, MIS), (7, A + 2, MIS), (8, 0, BAD),
                     (9, 0, BAD), (9, A + 4, MIS), (10, 0, BAD), (10, A + 8, MIS)):
        bad = list(ok)
        bad[i] = v
        refused(st, compute.gated_backward, *bad, **kw)
    refused(BAD, compute.gated_backward, *ok, workspace_bytes=n - 1)
    for ld in ("ld_dh", "ld_x", "ld_dx"):
        refused(BAD, compute.gated_backward, *ok, **kw, **{ld: 100})
    refused(BAD, compute.gated_backward, *ok, **kw, h=A, ld_h=100)
    ck = tide.GatedCheckpoint(A, A, A, A)
    bad = list(ok)
    bad[4] = 0  # weight gradients need the input
    refused(BAD, compute.gated_backward, *bad, **kw, checkpoint=ck)
    compute.gated_backward(0, 128, 256, 0, 0, A, A, 0, 0, 0, 0, workspace_bytes=0)


def test_null_handle_refused():
    lib = tide.tide._lib
    assert lib.tide_compute_create(None) == BAD
    assert lib.tide_fp8_store(None, 1, 1, A, 1, A, A, 1, None) == BAD
    assert lib.tide_fp8_restore(None, 1, 1, A, A, 1, A, 1, None) == BAD
    assert lib.tide_fp8_matmul(None, 1, 1, 1, A, A, A, A, 0, A, 1, None) == BAD
    assert lib.tide_gated_forward(None, 1, 1, 1, 0, A, 1, A, A, A, 1, None, None) == BAD
    assert lib.tide_gated_backward(None, 1, 1, 1, 0, A, 1, A, 1, A, A, None, A, 1, A, A, None, 1, A, 1 << 20, None) == BAD
    assert lib.tide_gated_workspace(1, 1, 1, None) == BAD
    lib.tide_compute_destroy(None)


def test_workspace_holds_its_parts():
    for m, k, f in ((1, 1, 1), (37, 2048, 768), (4093, 8192, 28672), (0, 5, 5)):
        assert tide.gated_workspace_bytes(m, k, f) >= 4 * m * f + 2 * m * k
    with pytest.raises(tide.TideError):
        tide.gated_workspace_bytes(-1, 1, 1)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_formulas_against_differences(kind):
    """The 64-bit gradients are the differences of the 64-bit forward pass."""
    g = torch.Generator().manual_seed(3)
    m, k, f = 3, 5, 4
    x, wg, wu, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((m, k), (f, k), (f, k), (m, f)))
    _, gg, uu = ref.gated_forward(x, wg, wu, kind)
    got = ref.gated_backward_from(dh, gg, uu, x, wg, wu, kind)[:3]
    step = 1e-6
    for t, grad in zip((x, wg, wu), got):
        for i in range(t.shape[0]):
            for j in range(t.shape[1]):
                keep = float(t[i, j])
                side = []
                for s in (step, -step):
                    t[i, j] = keep + s
                    side.append(float((dh * ref.gated_forward(x, wg, wu, kind)[0]).sum()))
                t[i, j] = keep
                # central difference: error ~ step^2 f''' + 2^-53 / step
                assert abs((side[0] - side[1]) / (2 * step) - float(grad[i, j])) < 1e-7


def test_checkpoint_struct_matches_header():
    assert ctypes.sizeof(tide.tide.GatedCheckpointStruct) == 6 * ctypes.sizeof(ctypes.c_void_p)


def test_test_hooks_refuse(compute):
    lib = tide.tide._lib
    for hook in (lib.tide_compute_set_test_stall, lib.tide_compute_set_test_late_warp):
        assert hook(None, 0) == BAD
        assert hook(compute.handle, -1) == BAD
        assert hook(compute.handle, 0) == tide.TIDE_OK


class Number:
    """A whole number that is no int."""

    def __init__(self, v):
        self.v = v

    def __int__(self):
        return self.v


@pytest.mark.parametrize("number", [Number, numpy.int64, numpy.uint64])
def test_tensors_and_streams_of_other_libraries(compute, number):
    """A buffer's data_ptr() and a stream's cuda_stream may be any whole number."""

    class Buffer:
        def data_ptr(self):
            return number(A)

    class Stream:
        cuda_stream = number(0)

    b, s = Buffer(), Stream()
    compute.fp8_store(0, 128, b, b, b, stream=s)
    refused(MIS, compute.fp8_store, 4, 128, b, b, A + 2, stream=s)
    with tide.Layout([], 2) as layout:
        layout.place(b, [], stream=s)
    with tide.Layout([(0, 4)], 2) as layout:
        layout.place(b, [b], stream=s)
