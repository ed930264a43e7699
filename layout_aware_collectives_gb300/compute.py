"""Owning wrapper around a tide_compute_t handle: the operators of the
feed-forward unit between a placement and the reduce-scatter, and of an expert
layer around it (marshalling only)."""
from __future__ import annotations

from . import tide as _t


class GatedCheckpoint:
    """Buffers of a gated block's activations in 8-bit blocks (1 x 128):
    codes [tokens, ffn] and scales [tokens, ceil(ffn / 128)] of the gate and up
    pre-activations and, where given, codes and scales of the input."""

    def __init__(self, gate_codes, gate_scales, up_codes, up_scales, x_codes=None, x_scales=None):
        self.keep = (gate_codes, gate_scales, up_codes, up_scales, x_codes, x_scales)
        self.struct = _t.GatedCheckpointStruct(*(_t._addr(b) for b in self.keep))


class Router:
    """How tokens choose their experts (tide_router_t); see include/tide.h."""

    def __init__(self, experts: int, topk: int, score: str = "softmax", groups: int = 1, top_groups: int = 1,
                 group_best: int = 1, renormalize: bool = True, scale: float = 1.0):
        self.experts, self.topk = experts, topk
        self.struct = _t.RouterStruct(experts, topk, _t._named(_t._SCORES, score, "score"), groups, top_groups,
                                      group_best, 1 if renormalize else 0, scale)


def _bytes(workspace, given):
    """A tensor's own size where it is left out; an address has none."""
    return workspace.numel() * workspace.element_size() if given is None else given


class Compute:
    """Operators of the feed-forward unit and the expert layer; see include/tide.h.

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
        workspace_bytes = _bytes(workspace, workspace_bytes)
        _t.tide_gated_backward(self.handle, tokens, hidden, ffn, activation, dh, ffn if ld_dh is None else ld_dh, x,
                               hidden if ld_x is None else ld_x, w_gate, w_up, checkpoint, dx,
                               hidden if ld_dx is None else ld_dx, dw_gate, dw_up, h, ffn if ld_h is None else ld_h,
                               workspace, workspace_bytes, stream)

    # -------- the expert layer
    def route(self, router: Router, tokens: int, logits, ids, weights, bias=None, logits_type: str | None = None,
              ld_logits=None, stream=None):
        """logits_type: "bf16" or "fp32"; a tensor's own where it is left out,
        fp32 of an address.  Tensors of other types than an operator reads or
        writes are refused (TypeError), here and in the other calls."""
        _t.tide_route(self.handle, tokens, router, logits_type, logits,
                      router.experts if ld_logits is None else ld_logits, bias, ids, weights, stream)

    def route_backward(self, router: Router, tokens: int, logits, ids, dweights, dlogits,
                       logits_type: str | None = None, ld_logits=None, ld_dlogits=None, stream=None):
        """logits_type: as in route, dlogits' too."""
        _t.tide_route_backward(self.handle, tokens, router, logits_type, logits,
                               router.experts if ld_logits is None else ld_logits, ids, dweights, dlogits,
                               router.experts if ld_dlogits is None else ld_dlogits, stream)

    def expert_slots(self, tokens: int, topk: int, experts: int, ids, slots, offsets, workspace, workspace_bytes=None,
                     stream=None):
        """workspace_bytes: as in gated_backward."""
        _t.tide_expert_slots(self.handle, tokens, topk, experts, ids, slots, offsets, workspace,
                             _bytes(workspace, workspace_bytes), stream)

    def expert_gather(self, tokens: int, hidden: int, topk: int, x, slots, rows, num_rows: int, ld_x=None, ld_rows=None,
                      stream=None):
        _t.tide_expert_gather(self.handle, tokens, hidden, topk, x, hidden if ld_x is None else ld_x, slots, rows,
                              num_rows, hidden if ld_rows is None else ld_rows, stream)

    def expert_combine(self, tokens: int, hidden: int, topk: int, rows, num_rows: int, slots, weights, y, ld_rows=None,
                       ld_y=None, stream=None):
        _t.tide_expert_combine(self.handle, tokens, hidden, topk, rows, num_rows,
                               hidden if ld_rows is None else ld_rows, slots, weights, y,
                               hidden if ld_y is None else ld_y, stream)

    def expert_combine_backward(self, tokens: int, hidden: int, topk: int, dy, rows, num_rows: int, slots, weights,
                                drows, dweights, ld_dy=None, ld_rows=None, ld_drows=None, stream=None):
        _t.tide_expert_combine_backward(self.handle, tokens, hidden, topk, dy, hidden if ld_dy is None else ld_dy, rows,
                                        num_rows, hidden if ld_rows is None else ld_rows, slots, weights, drows,
                                        hidden if ld_drows is None else ld_drows, dweights, stream)

    def orthogonalize(self, rows: int, cols: int, src, dst, workspace, steps: int = 5, coefficients=None,
                      eps: float = 1e-7, src_type: str | None = None, workspace_bytes=None, ld_src=None, ld_dst=None,
                      stream=None):
        """src, dst: lists of matrices of one size; src_type: as logits_type in
        route; workspace_bytes: as in gated_backward."""
        _t.tide_orthogonalize(self.handle, rows, cols, src_type, src, cols if ld_src is None else ld_src, dst,
                              cols if ld_dst is None else ld_dst, steps, coefficients, eps, workspace,
                              _bytes(workspace, workspace_bytes), stream)

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
