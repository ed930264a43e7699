"""Owning wrapper around a tide_compute_t handle: the feed-forward unit's
operators between a placement and the reduce-scatter (marshalling only)."""
from __future__ import annotations

from . import tide as _t


class GatedCheckpoint:
    """Buffers of a gated block's activations in 8-bit blocks (1 x 128):
    codes [tokens, ffn] and scales [tokens, ceil(ffn / 128)] of the gate and up
    pre-activations and, where given, codes and scales of the input."""

    def __init__(self, gate_codes, gate_scales, up_codes, up_scales, x_codes=None, x_scales=None):
        self.keep = (gate_codes, gate_scales, up_codes, up_scales, x_codes, x_scales)
        self.struct = _t.GatedCheckpointStruct(*(_t._addr(b) for b in self.keep))


class Compute:
    """Feed-forward operators; see include/tide.h.

    Row strides (ld_*) default to the row's width."""

    def __init__(self):
        self.handle = _t.tide_compute_create()

    def fp8_store(self, rows: int, cols: int, src, codes, scales, block_rows: int = 1, ld_src=None, stream=None):
        _t.tide_fp8_store(self.handle, rows, cols, src, cols if ld_src is None else ld_src, codes, scales, block_rows,
                          stream)

    def fp8_restore(self, rows: int, cols: int, codes, scales, dst, block_rows: int = 1, ld_dst=None, stream=None):
        _t.tide_fp8_restore(self.handle, rows, cols, codes, scales, block_rows, dst, cols if ld_dst is None else ld_dst,
                            stream)

    def fp8_matmul(self, m: int, n: int, k: int, a, a_scales, b, b_scales, out, any_scales: bool = False, ld_out=None,
                   stream=None):
        """any_scales: scales other than the powers of two that fp8_store writes."""
        _t.tide_fp8_matmul(self.handle, m, n, k, a, a_scales, b, b_scales, any_scales, out,
                           n if ld_out is None else ld_out, stream)

    def gated_forward(self, tokens: int, hidden: int, ffn: int, x, w_gate, w_up, h, activation: str = "silu",
                      checkpoint: GatedCheckpoint | None = None, ld_x=None, ld_h=None, stream=None):
        _t.tide_gated_forward(self.handle, tokens, hidden, ffn, activation, x, hidden if ld_x is None else ld_x, w_gate,
                              w_up, h, ffn if ld_h is None else ld_h, checkpoint, stream)

    def gated_backward(self, tokens: int, hidden: int, ffn: int, dh, x, w_gate, w_up, dx, dw_gate, dw_up, workspace,
                       activation: str = "silu", checkpoint: GatedCheckpoint | None = None, h=None,
                       workspace_bytes=None, ld_dh=None, ld_x=None, ld_dx=None, ld_h=None, stream=None):
        """workspace_bytes: a tensor's own size where it is left out; to be
        given with an address."""
        if workspace_bytes is None:
            workspace_bytes = workspace.numel() * workspace.element_size()
        _t.tide_gated_backward(self.handle, tokens, hidden, ffn, activation, dh, ffn if ld_dh is None else ld_dh, x,
                               hidden if ld_x is None else ld_x, w_gate, w_up, checkpoint, dx,
                               hidden if ld_dx is None else ld_dx, dw_gate, dw_up, h, ffn if ld_h is None else ld_h,
                               workspace, workspace_bytes, stream)

    def check_device(self) -> None:
        _t.tide_compute_check_device(self.handle)

    def set_test_stall(self, ns: int) -> None:
        _t.tide_compute_set_test_stall(self.handle, ns)

    def set_test_late_warp(self, ns: int) -> None:
        _t.tide_compute_set_test_late_warp(self.handle, ns)

    # -------- lifetime
    def close(self) -> None:
        if getattr(self, "handle", None):
            _t.tide_compute_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
