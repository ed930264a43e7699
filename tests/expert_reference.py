"""Plain 64-bit definitions of the expert layer's operators, and error bounds.

Every bound is derived from the formats: a rounding is off by at most half a
step (bf16 2^-8 of the value, fp16 2^-11, fp32 2^-24), exp of an argument off by
d is off by d of itself, and a sum of k fp32 terms by at most (k + 8) 2^-24 of
its terms' magnitudes.
"""
import math

import torch

U_BF16 = 2.0 ** -8
U_F16 = 2.0 ** -11
U_F32 = 2.0 ** -24
TINY = 2.0 ** -126
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def scores(logits, score):
    """Softmax or sigmoid in 64 bits; masked experts (-infinity) have 0."""
    l = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    top = l.amax(1, keepdim=True)
    e = torch.where(l == -math.inf, torch.zeros_like(l), torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = e.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def shares(logits, score):
    """Scores over their sum, of the chosen experts' logits alone.  Sigmoids by
    their logarithms: far below zero 64 bits do not hold them, but their ratios."""
    log = logits.double() if score == "softmax" else torch.nn.functional.logsigmoid(logits.double())
    top = log.amax(1, keepdim=True)
    e = torch.where(log == -math.inf, torch.zeros_like(log), torch.exp(log - torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = e.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def _ranked(v, k):
    """Indices of the k largest; NaN below everything, the lowest of equals first."""
    order = torch.where(torch.isnan(v), torch.full_like(v, -math.inf), v)
    # NaN after -infinity: two stable sorts
    first = torch.sort(torch.isnan(v).int(), dim=1, stable=True).indices
    second = torch.sort(order.gather(1, first), dim=1, descending=True, stable=True).indices
    return first.gather(1, second)[:, :k]


def route(logits, topk, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(ids, weights) of the definition."""
    t, e = logits.shape
    s = scores(logits, score)
    if bias is not None or (groups > 1 and group_best == 2 and e // groups > 1):
        c = s if bias is None else s + bias.double()
    else:
        c = logits.double()  # scores grow with logits
    c = c.clone()
    if groups > 1:
        each = e // groups
        by = c.view(t, groups, each)
        best = by.gather(2, _ranked(by.reshape(t * groups, each), min(group_best, each)).view(t, groups, -1)).sum(2)
        kept = _ranked(best, top_groups)
        out = torch.ones(t, groups, dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        # behind every expert of a kept group, NaN among them
        mask = out.repeat_interleave(each, 1)
        key = torch.where(torch.isnan(c), torch.full_like(c, -math.inf), c)
        stay = torch.sort(mask.int(), dim=1, stable=True).indices
        inner = _ranked_with(key.gather(1, stay), torch.isnan(c).gather(1, stay).int() + 2 * mask.gather(1, stay).int())
        ids = stay.gather(1, inner)[:, :topk]
    else:
        ids = _ranked(c, topk)
    w = (shares(logits.gather(1, ids), score) if renormalize else s.gather(1, ids)) * scale
    if score == "softmax":
        bad = torch.isnan(logits).any(1) | (logits == math.inf).any(1)
        w[bad] = math.nan
    return ids, w


def _ranked_with(v, level):
    """Indices by level, then from the largest value, then by place."""
    a = torch.sort(v, dim=1, descending=True, stable=True).indices
    b = torch.sort(level.gather(1, a), dim=1, stable=True).indices
    return a.gather(1, b)


def route_bound(logits, ids, w, score):
    """|error| of weights: 128 roundings, and exp's argument l - top, or l."""
    l = logits.double()
    far = l.gather(1, ids).abs() if score == "sigmoid" else (l.gather(1, ids) - l.amax(1, keepdim=True)).abs()
    return (128 + 4 * torch.nan_to_num(far, nan=0.0, posinf=0.0).clamp(max=200)) * U_F32 * w.abs() + TINY * 2 ** 10


def route_backward(logits, ids, dweights, score, renormalize, scale):
    """dlogits by the formulas, and a bound of its |error|."""
    l = logits.double()
    t, e = l.shape
    s = scores(l, score)
    inside = (ids >= 0) & (ids < e)
    at = ids.long().clamp(0, e - 1)
    g = torch.where(inside, dweights.double() * scale, torch.zeros((), dtype=torch.float64, device=l.device))
    p = torch.where(inside, s.gather(1, at), torch.zeros_like(g))
    far = 4 * l.gather(1, at).abs().clamp(max=200)
    if renormalize:
        p = shares(torch.where(inside, l.gather(1, at), torch.full_like(g, -math.inf)), score)
        mean = (p * g).sum(1, keepdim=True)
        rest = torch.sigmoid(-l.gather(1, at)) if score == "sigmoid" else 1.0
        each, size = p * (g - mean) * rest, p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    elif score == "sigmoid":
        each = g * p * torch.sigmoid(-l.gather(1, at))
        size = each.abs()
    else:
        d = torch.zeros_like(s).scatter_add_(1, at, torch.where(inside, g, torch.zeros_like(g)))
        a = torch.zeros_like(s).scatter_add_(1, at, g.abs())
        out = s * (d - (d * s).sum(1, keepdim=True))
        big = s * (a + (a * s).sum(1, keepdim=True))
        reach = torch.nan_to_num((l.amax(1, keepdim=True) - l).clamp(max=200))  # a row without experts has no reach
        return out, (256 + 8 * reach + e) * U_F32 * big + TINY * 2 ** 10
    zero = torch.zeros_like(s)
    out = zero.scatter_add(1, at, torch.where(inside, each, torch.zeros_like(each)))
    big = zero.scatter_add(1, at, torch.where(inside, (256 + 2 * far) * size, torch.zeros_like(size)))
    return out, big * U_F32 + TINY * 2 ** 10


def slots(ids, experts):
    """(slots, offsets): pairs by expert, then in their own order."""
    flat = ids.reshape(-1).long().cpu()
    out = torch.full_like(flat, -1)
    offsets, at = [0], 0
    for e in range(experts):
        mine = torch.nonzero(flat == e).reshape(-1)
        out[mine] = torch.arange(at, at + mine.numel())
        at += mine.numel()
        offsets.append(at)
    return out.view(ids.shape).int(), torch.tensor(offsets, dtype=torch.int32)


def combine(rows, slots, weights):
    """(y, bound): rows' mixtures in 64 bits; slots outside the rows are passed over."""
    t, k = slots.shape
    inside = (slots >= 0) & (slots < rows.shape[0])
    each = rows.double()[slots.long().clamp(0, rows.shape[0] - 1)] * inside[:, :, None]
    w = torch.ones(t, k, dtype=torch.float64, device=rows.device) if weights is None else weights.double()
    y = (each * w[:, :, None]).sum(1)
    off = (k + 8) * U_F32 * (each.abs() * w.abs()[:, :, None]).sum(1)
    return y, off + U_BF16 * (y.abs() + off) + TINY


def combine_backward(dy, rows, slots, weights):
    """(drows' values for each pair, bound, dweights, bound)."""
    t, k = slots.shape
    inside = (slots >= 0) & (slots < rows.shape[0])
    each = rows.double()[slots.long().clamp(0, rows.shape[0] - 1)] * inside[:, :, None]
    w = torch.ones(t, k, dtype=torch.float64, device=rows.device) if weights is None else weights.double()
    d = dy.double()[:, None, :]
    drows = w[:, :, None] * d
    dw = (d * each).sum(2)
    return drows, (U_BF16 + 2 * U_F32) * drows.abs() + TINY, dw, (dy.shape[1] + 8) * U_F32 * (d * each).abs().sum(2) + TINY


def orthogonalize(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """X of the definition, in 64 bits."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    x = x / (x.norm() + eps)
    for i in range(steps):
        a, b, c = step_of(coefficients, i)
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if tall else x


def step_of(coefficients, i):
    c = [float(torch.tensor(v, dtype=torch.float32)) for v in coefficients]
    return c if len(c) == 3 else c[3 * i:3 * i + 3]


def orthogonalize_bound(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """A bound of the error's Frobenius norm, before the rounding to bf16.

    The roundings that the operator allows itself (X as two fp16 terms, of which
    products take the first; the symmetric matrices as one beside their diagonals;
    two steps by one pass over X where rows and columns allow it) are made here in
    64 bits, and three times what they leave is allowed: other roundings of the same
    sizes leave as much, not more, and fp32's own are 2^13 times smaller.  fp16's
    smallest numbers leave out what is below 2^-37 of the largest norm that X can
    have; every step stretches that by at most the largest slope of s -> s (a + b
    s^2 + c s^4) for singular values from 0 on."""
    want = orthogonalize(g, steps, coefficients, eps)
    off = max(float((_rounded(g, steps, coefficients, eps, pairs) - want).norm()) for pairs in (False, True))
    stretch, bound, floor = 1.0, 1.0, 2.0 ** -37
    for i in range(steps):
        a, b, c = step_of(coefficients, i)
        s = torch.linspace(0, bound, 4001, dtype=torch.float64)
        stretch = max(1.0, float(torch.maximum((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs(), (a + b * s ** 2 + c * s ** 4).abs()).max()))
        bound = float((a * s + b * s ** 3 + c * s ** 5).abs().max())
        floor = stretch * floor + bound * 2.0 ** -37
    return 3 * off + floor * math.sqrt(g.numel())


class _Kept:
    """A symmetric matrix as one fp16 term, its diagonal beside it."""

    def __init__(self, v):
        self.d = v.diagonal().clone()
        self.p = _half(v - torch.diag(self.d))

    def __matmul__(self, o):
        v = self.p @ o.p + self.d[:, None] * o.p + self.p * o.d[None, :] + torch.diag(self.d * o.d)
        return (v + v.T) / 2

    def value(self):
        return self.p + torch.diag(self.d)


def _half(v):
    """Rounded to fp16 of a power-of-two scale that brings the largest to 2^13."""
    top = float(v.abs().max()) if v.numel() else 0.0
    if top == 0 or not math.isfinite(top):
        return v
    scale = 2.0 ** (13 - math.ceil(math.log2(top)))
    return (v * scale).half().double() / scale


def _rounded(g, steps, coefficients, eps, pairs):
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    x = x / (x.norm() + eps)
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    i = 0
    while i < steps:
        hi = _half(x)
        x = hi + _half(x - hi)
        a, b, c = step_of(coefficients, i)
        gram = _Kept(hi @ hi.T)
        poly = _Kept(a * eye + b * gram.value() + c * (gram @ gram))
        i += 1
        if pairs and i < steps:
            a, b, c = step_of(coefficients, i)
            second = _Kept(_Kept(poly @ gram) @ poly)
            poly = _Kept(_Kept(a * eye + b * second.value() + c * (second @ second)) @ poly)
            i += 1
        x = poly.p @ hi + poly.d[:, None] * x
    return x.T if tall else x
