"""Plain 64-bit definitions of the feed-forward operators, and error bounds.

Every bound is derived from the formats: 2^-8 is bf16's largest relative
rounding error, a k-term fp32 sum in any order is off by at most
(k + 8) 2^-23 of the sum of its terms' magnitudes (truncating adders counted),
and the activations and their derivatives have slopes below 1.2.
"""
import math

import torch

U_BF16 = 2.0 ** -8
U_F32 = 2.0 ** -23
TINY = 2.0 ** -126  # fp32 results below the normal range may be flushed


def blocks_store(v, block_rows):
    """(codes float8_e4m3fn, scales float32) of a float32 matrix, by the definition."""
    r, c = v.shape
    nr, nc = -(-r // block_rows), -(-c // 128)
    codes = torch.empty(r, c, dtype=torch.float8_e4m3fn, device=v.device)
    scales = torch.ones(nr, nc, dtype=torch.float32, device=v.device)
    for i in range(nr):
        for j in range(nc):
            b = v[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            f = b[torch.isfinite(b)].abs()
            s = 1.0
            if f.numel() and f.max() > 0:
                s = 2.0 ** max(-126, math.ceil(math.log2(float(f.max())) - math.log2(448)))
                while s > 2.0 ** -126 and float(f.max()) <= 448 * (s / 2):  # log2 near an exact power
                    s /= 2
                while float(f.max()) > 448 * s:
                    s *= 2
            scales[i, j] = s
            q = torch.where(torch.isfinite(b), b / s, torch.full_like(b, math.nan))
            codes[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128] = q.to(torch.float8_e4m3fn)
    return codes, scales


def blocks_value(codes, scales, block_rows):
    """The values of 8-bit blocks in 64 bits."""
    i = torch.arange(codes.shape[0], device=codes.device) // block_rows
    j = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.float().double() * scales.double()[i][:, j]


def act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(2 * z)  # 0.5 (1 + tanh z), without its cancellation


def act_grad(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s, r = torch.sigmoid(2 * z), torch.sigmoid(-2 * z)
    return s + 2 * g * s * r * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def arithmetic(g, kind):
    """Relative rounding of the activations' own fp32 arithmetic: 32 roundings,
    and an exponential whose argument e is off by up to 4 2^-23 of itself."""
    e = g.abs() if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3).abs()
    return (32 + 8 * e.clamp(max=200)) * U_F32


def flushed(g):
    """What is left out where the sigmoid falls below the normal range."""
    return TINY * (1 + g.abs().clamp(max=100)) ** 3


def gated_forward(x, wg, wu, kind):
    """h, g, u in 64 bits."""
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    return act(g, kind) * u, g, u


def gated_forward_bound(x, wg, wu, kind):
    """Bounds of |error| of h, g and u."""
    h, g, u = gated_forward(x, wg, wu, kind)
    k = x.shape[1]
    eg = (k + 8) * U_F32 * (x.double().abs() @ wg.double().abs().T)
    eu = (k + 8) * U_F32 * (x.double().abs() @ wu.double().abs().T)
    a = act(g, kind).abs()
    ea = 1.2 * eg + a * arithmetic(g, kind) + flushed(g)
    eh = u.abs() * ea + a * eu + ea * eu
    return eh + U_BF16 * (h.abs() + eh) + TINY, eg + TINY, eu + TINY


def gated_backward_from(dh, g, u, x, wg, wu, kind):
    """dx, dWg, dWu, h in 64 bits from the pre-activations."""
    dh, x = dh.double(), x.double()
    du, dg = dh * act(g, kind), dh * u * act_grad(g, kind)
    return dg @ wg.double() + du @ wu.double(), dg.T @ x, du.T @ x, act(g, kind) * u


def gated_backward_bound(dh, g, u, x, wg, wu, kind, eg=0.0, eu=0.0):
    """Bounds of |error| of dx, dWg, dWu when g and u are off by up to eg, eu."""
    dh, x = dh.double(), x.double()
    a, d = act(g, kind), act_grad(g, kind)
    arith = arithmetic(g, kind)
    ea = 1.2 * eg + a.abs() * arith + flushed(g)
    # the derivative is a sum of terms up to 1 + 2 |g| s (1 - s) dz < 3 that may cancel
    ed = 1.2 * eg + 3 * (32 + 8 * 20) * U_F32 + flushed(g)
    du, dg = dh * a, dh * u * d
    edu = dh.abs() * ea
    edg = dh.abs() * (u.abs() * ed + d.abs() * eu + ed * eu)
    edu = edu + U_BF16 * (du.abs() + edu) + TINY
    edg = edg + U_BF16 * (dg.abs() + edg) + TINY
    m, f = dh.shape

    def product(e, v, w, terms):
        return e @ w.abs() + (terms + 8) * U_F32 * ((v.abs() + e) @ w.abs())

    wg, wu = wg.double(), wu.double()
    bx = product(edg, dg, wg, 2 * f) + product(edu, du, wu, 2 * f)
    bg, bu = product(edg.T, dg.T, x, m), product(edu.T, du.T, x, m)
    dx, dwg, dwu, _ = gated_backward_from(dh, g, u, x, wg, wu, kind)
    return tuple(b + U_BF16 * (r.abs() + b) + TINY for b, r in ((bx, dx), (bg, dwg), (bu, dwu)))


def matmul(a, sa, b, sb):
    """(value, bound of |error|) of the product of two matrices in 8-bit blocks."""
    av, bv = blocks_value(a, sa, 1), blocks_value(b, sb, 128)
    r = av @ bv.T
    e = (a.shape[1] + 8) * U_F32 * (av.abs() @ bv.abs().T)
    return r, e + U_BF16 * (r.abs() + e) + TINY
