"""The operators at the two ends of an expert layer's training step.

Its router's logits decide which tokens an expert's gated block gets; the tokens
are brought to the experts and their results back; and the weights' gradients,
which the reduce-scatter delivers matrix by matrix, become updates:

  route           ids and weights of each token's experts from its logits
  route_backward  the logits' gradients from the weights'
  dispatch        each (token, expert) pair's row in expert order, and the
                  tokens' rows copied there
  combine         a token's results from its experts' rows, by their weights
  combine_backward   the rows' and the weights' gradients
  orthogonalize   Newton-Schulz products: the orthogonal factor of an update

`run` computes them in plain torch operations in 32 bits (selections in 64), or,
with `own`, by the framework's kernels.
"""
import math

import torch

own = False

_handle = None


def _compute():
    """The handle that a program keeps for all its calls."""
    global _handle
    if _handle is None:
        import layout_aware_collectives_gb300 as tide

        _handle = tide.Compute()
    return _handle


COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ---------------------------------------------------------------- the cases

def _route(kind, tokens, experts, topk, score, dtype, bias=False, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    return dict(kind=kind, tokens=tokens, experts=experts, topk=topk, score=score, dtype=dtype, bias=bias, groups=groups,
                top_groups=top_groups, best=best, renorm=renorm, scale=scale)


def listed():
    return [
        # one generated token through the 128-expert layer's router
        dict(_route("route", 1, 128, 8, "softmax", "float32"), name="route_token"),
        # a training step's tokens, balanced by a bias, in groups of experts
        dict(_route("route", 8192, 256, 8, "sigmoid", "float32", bias=True, groups=8, top_groups=4, best=2, scale=2.5),
             name="route_groups_8192"),
        # the 128-expert layer's backward pass, weights as the softmax gave them
        dict(_route("route_backward", 8192, 128, 8, "softmax", "bfloat16", renorm=False), name="route_backward_8192"),
        # a ragged batch's backward pass, an odd number of experts
        dict(_route("route_backward", 1021, 60, 4, "sigmoid", "float32"), name="route_backward_1021"),
        # a ragged handful of tokens to the 128-expert layer
        dict(kind="dispatch", tokens=37, hidden=2048, topk=8, experts=128, name="dispatch_37"),
        # a training step's tokens to the 128-expert layer, one short of a power of two
        dict(kind="dispatch", tokens=8191, hidden=2048, topk=8, experts=128, name="dispatch_8191"),
        # a 4096-wide layer's results back, two experts a token
        dict(kind="combine", tokens=4096, hidden=4096, topk=2, experts=8, name="combine_4096"),
        # the 128-expert layer's backward pass of an odd number of tokens
        dict(kind="combine_backward", tokens=4093, hidden=2048, topk=8, experts=128, name="combine_backward_4093"),
        # the tiny block's gate projection
        dict(kind="orthogonalize", count=1, rows=704, cols=256, dtype="float32", name="orthogonalize_tiny"),
        # a few matrices of odd sizes
        dict(kind="orthogonalize", count=3, rows=1021, cols=1375, dtype="float32", name="orthogonalize_odd"),
        # the gate projections of the 128-expert layer, as they were placed
        dict(kind="orthogonalize", count=128, rows=768, cols=2048, dtype="bfloat16", name="orthogonalize_experts"),
        # the 8B-shaped layer's gate projection
        dict(kind="orthogonalize", count=1, rows=14336, cols=4096, dtype="float32", name="orthogonalize_8b"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route", "route_backward", "dispatch", "combine", "combine_backward", "orthogonalize", "orthogonalize"])
    tokens, topk = _log(rng, 1, 8192), rng.randint(1, 10)
    if kind in ("route", "route_backward"):
        score, dtype = rng.choice(["softmax", "sigmoid"]), rng.choice(["float32", "bfloat16"])
        groups = rng.choice([1, 1, 2, 4, 8])
        each = _log(rng, 10, 512 // groups)
        top = rng.randint(max(1, groups // 2), groups)
        topk = min(max(2, topk), top * each)  # one renormalised weight has no gradient
        return _route(kind, tokens, groups * each, topk, score, dtype, bias=kind == "route" and rng.random() < 0.5, groups=groups,
                      top_groups=top, best=rng.choice([1, 2]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if kind == "orthogonalize":
        rows, cols = _log(rng, 32, 4096), _log(rng, 32, 4096)
        small = min(rows, cols) ** 2 * max(rows, cols)
        return dict(kind=kind, count=min(_log(rng, 1, 64), max(1, 10 ** 11 // small)), rows=rows, cols=cols,
                    dtype=rng.choice(["float32", "bfloat16"]))
    # every other width is odd
    hidden = _log(rng, 64, 8192)
    hidden = hidden | 1 if rng.random() < 0.5 else (hidden + 7) // 8 * 8
    tokens = min(tokens, max(1, (1 << 27) // (hidden * topk)))
    return dict(kind=kind, tokens=tokens, hidden=hidden, topk=topk, experts=_log(rng, 10, 512))


def work(case):
    c = case
    if c["kind"] == "orthogonalize":
        m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # two of the three products are symmetric: half of each is the other half
        each = STEPS * (m * m * n + m * m * m + 2 * m * m * n)
        return {"bytes": c["count"] * m * n * (6 if c["dtype"] == "float32" else 4), "flops": c["count"] * each}
    t, k, e = c["tokens"], c["topk"], c["experts"]
    if c["kind"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": t * e * size + 8 * t * k + (4 * e if c["bias"] else 0), "flops": 4 * t * e}
    if c["kind"] == "route_backward":
        size = 4 if c["dtype"] == "float32" else 2
        # renormalised weights go by their own logits alone
        read = t * (k if c["renorm"] or c["score"] == "sigmoid" else e)
        return {"bytes": (read + t * e) * size + 8 * t * k, "flops": 6 * read}
    h = c["hidden"]
    if c["kind"] == "dispatch":
        return {"bytes": 8 * t * k + 4 * (e + 1) + 2 * t * h + 2 * t * k * h, "flops": t * k}
    if c["kind"] == "combine":
        return {"bytes": 8 * t * k + 2 * t * k * h + 2 * t * h, "flops": 2 * t * k * h}
    return {"bytes": 12 * t * k + 2 * t * h + 4 * t * k * h, "flops": 3 * t * k * h}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _logits(g, tokens, experts, dtype):
    """A token's own preferences, and some experts liked by all."""
    return (_randn(g, tokens, experts, scale=1.5) + _randn(g, experts, scale=0.5)).to(dtype)


def _choice(g, tokens, experts, topk):
    """Each token's experts, distinct, some experts more often than others."""
    return torch.topk(_randn(g, tokens, experts) + _randn(g, experts, scale=0.5), topk, dim=1).indices.int()


def _order(ids, experts):
    """(row of each pair in expert order, first row of each expert and the end)."""
    flat = ids.reshape(-1).long()
    at = torch.argsort(flat, stable=True)
    slots = torch.empty_like(at)
    slots[at] = torch.arange(at.numel(), device=at.device)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=at.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(experts, device=at.device)).sum(0), 0)
    return slots.view(ids.shape).int(), offsets.int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["kind"] == "orthogonalize":
        # gradients: a few directions over a floor of noise, each matrix with its own size
        n, r, q = c["count"], c["rows"], c["cols"]
        grads = _randn(g, n, r, q)
        grads += torch.bmm(_randn(g, n, r, 4), _randn(g, n, 4, q))
        grads *= torch.exp(_randn(g, n, 1, 1)) * 1e-3
        s["grads"] = grads.to(getattr(torch, c["dtype"]))
        s["updates"] = new(n, r, q)
        return s
    t, k, e = c["tokens"], c["topk"], c["experts"]
    if c["kind"] in ("route", "route_backward"):
        dtype = getattr(torch, c["dtype"])
        s["logits"] = _logits(g, t, e, dtype)
        if c["kind"] == "route":
            s["bias"] = _randn(g, e, scale=0.05) if c["bias"] else None
            s.update(ids=new(t, k, dtype=torch.int32), weights=new(t, k, dtype=torch.float32))
        else:
            s["ids"] = torch.topk(s["logits"].float(), k, dim=1).indices.int()
            s.update(dweights=_randn(g, t, k), dlogits=new(t, e, dtype=dtype))
        return s
    h = c["hidden"]
    s["ids"] = _choice(g, t, e, k)
    if c["kind"] == "dispatch":
        s.update(x=_randn(g, t, h).bfloat16(), rows=new(t * k, h), slots=new(t, k, dtype=torch.int32), offsets=new(e + 1, dtype=torch.int32))
        return s
    s["slots"] = _order(s["ids"], e)[0]
    s["rows"] = _randn(g, t * k, h).bfloat16()
    s["weights"] = torch.softmax(_randn(g, t, k), dim=1)
    if c["kind"] == "combine":
        s["y"] = new(t, h)
    else:
        s.update(dy=_randn(g, t, h, scale=1.0 / 64).bfloat16(), drows=new(t * k, h), dweights=new(t, k, dtype=torch.float32))
    return s


# ---------------------------------------------------------------- one pass

def _scores(logits, score):
    """In the logits' own type."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _first_best(values, k):
    """Indices of the k largest of each row, in order; the lowest index of equals."""
    return torch.sort(values, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s, c):
    # borders between two experts are decided in 64 bits
    scores = _scores(s["logits"].double(), c["score"])
    choice = scores if s["bias"] is None else scores + s["bias"].double()
    if c["groups"] > 1:
        t, g = c["tokens"], c["groups"]
        best = torch.sort(choice.view(t, g, -1), dim=2, descending=True).values[:, :, :c["best"]].sum(2)
        keep = torch.zeros(t, g, dtype=torch.bool, device=choice.device)
        keep.scatter_(1, _first_best(best, c["top_groups"]), True)
        each = c["experts"] // g
        choice = torch.where(keep.repeat_interleave(each, 1), choice, torch.full_like(choice, -math.inf))
    ids = _first_best(choice, c["topk"])
    w = scores.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * c["scale"]).float()


def _plain_route_backward(s, c):
    scores = _scores(s["logits"].float(), c["score"])
    ids, g = s["ids"].long(), s["dweights"] * c["scale"]
    picked = scores.gather(1, ids)
    if c["renorm"]:
        # w = s / sum(s): the weights' gradients become the scores'
        total = picked.sum(1, keepdim=True)
        g = (g - (g * picked).sum(1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        rest = 1 / (1 + torch.exp(s["logits"].float().gather(1, ids)))  # 1 - picked, without its cancellation
        d = torch.zeros_like(scores).scatter_(1, ids, g * picked * rest)
    else:
        d = torch.zeros_like(scores).scatter_(1, ids, g)
        d = scores * (d - (g * picked).sum(1, keepdim=True))
    return d.to(s["dlogits"].dtype)


def _plain_orthogonalize(s, c):
    x = s["grads"].float()
    tall = c["rows"] > c["cols"]
    if tall:
        x = x.mT
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x / (norm + EPS)).float()
    a, b, q = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + q * (gram @ gram)) @ x
    return (x.mT if tall else x).bfloat16()


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "route":
        return _plain_route(s, c)
    if kind == "route_backward":
        return _plain_route_backward(s, c)
    if kind == "orthogonalize":
        return _plain_orthogonalize(s, c)
    t, k = c["tokens"], c["topk"]
    if kind == "dispatch":
        slots, offsets = _order(s["ids"], c["experts"])
        rows = torch.empty_like(s["rows"])
        rows[slots.reshape(-1).long()] = s["x"].repeat_interleave(k, 0)
        return slots, offsets, rows
    at = s["slots"].reshape(-1).long()
    each = s["rows"][at].float().view(t, k, -1)
    if kind == "combine":
        return (each * s["weights"][:, :, None]).sum(1).bfloat16()
    dy = s["dy"].float()[:, None, :]
    drows = torch.empty_like(s["rows"])
    drows[at] = (dy * s["weights"][:, :, None]).bfloat16().view(t * k, -1)
    return drows, (dy * each).sum(2)


def _run_own(s):
    import layout_aware_collectives_gb300 as tide

    c, o, stream = s["case"], _compute(), torch.cuda.current_stream()
    kind = c["kind"]
    new = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    if kind == "orthogonalize":
        r, q = c["rows"], c["cols"]
        if "tables" not in s:
            s["tables"] = tide.PointerTable(s["grads"].unbind(0)), tide.PointerTable(s["updates"].unbind(0))
            s["workspace"] = new(tide.orthogonalize_workspace_bytes(c["count"], r, q))
        o.orthogonalize(r, q, *s["tables"], s["workspace"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                        src_type="fp32" if c["dtype"] == "float32" else "bf16", stream=stream)
        return s["updates"]
    t, k, e = c["tokens"], c["topk"], c["experts"]
    if kind in ("route", "route_backward"):
        if "router" not in s:
            s["router"] = tide.Router(e, k, score=c["score"], groups=c["groups"], top_groups=c["top_groups"], group_best=c["best"],
                                      renormalize=c["renorm"], scale=c["scale"])
        logits_type = "fp32" if c["dtype"] == "float32" else "bf16"
        if kind == "route":
            o.route(s["router"], t, s["logits"], s["ids"], s["weights"], bias=s["bias"], logits_type=logits_type, stream=stream)
            return s["ids"], s["weights"]
        o.route_backward(s["router"], t, s["logits"], s["ids"], s["dweights"], s["dlogits"], logits_type=logits_type, stream=stream)
        return s["dlogits"]
    h = c["hidden"]
    if kind == "dispatch":
        if "workspace" not in s:
            s["workspace"] = new(tide.expert_slots_workspace_bytes(t, k, e))
        o.expert_slots(t, k, e, s["ids"], s["slots"], s["offsets"], s["workspace"], stream=stream)
        o.expert_gather(t, h, k, s["x"], s["slots"], s["rows"], t * k, stream=stream)
        return s["slots"], s["offsets"], s["rows"]
    if kind == "combine":
        o.expert_combine(t, h, k, s["rows"], t * k, s["slots"], s["weights"], s["y"], stream=stream)
        return s["y"]
    o.expert_combine_backward(t, h, k, s["dy"], s["rows"], t * k, s["slots"], s["weights"], s["drows"], s["dweights"], stream=stream)
    return s["drows"], s["dweights"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, in 64 bits; None for whole numbers."""
    s, c = prepare(case, seed), case
    kind = c["kind"]
    if kind == "orthogonalize":
        x = s["grads"].double()
        x = x / (torch.linalg.matrix_norm(x, keepdim=True) + EPS)
        a, b, q = COEFFICIENTS
        for _ in range(STEPS):  # from the right where that is the shorter side
            gram = torch.matmul(x.mT, x) if c["rows"] > c["cols"] else torch.matmul(x, x.mT)
            poly = torch.matmul(gram, gram).mul_(q).add_(gram, alpha=b)
            poly.diagonal(dim1=1, dim2=2).add_(a)
            x = torch.matmul(x, poly) if c["rows"] > c["cols"] else torch.matmul(poly, x)
        return x
    t, k = c["tokens"], c["topk"]
    if kind in ("route", "route_backward"):
        logits = s["logits"].double()
        scores = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, 1)
        if kind == "route":
            choice = scores.clone() if s["bias"] is None else scores + s["bias"].double()
            each = c["experts"] // c["groups"]
            if c["groups"] > 1:
                by = choice.view(t, c["groups"], each)
                score = by.topk(min(c["best"], each), 2).values.sum(2)
                # a group's place: how many are above it, or equal and before it
                above = score[:, None, :] > score[:, :, None]
                at = torch.arange(c["groups"], device=score.device)
                above |= (score[:, None, :] == score[:, :, None]) & (at[None, :] < at[:, None])
                by[above.sum(2) >= c["top_groups"]] = -math.inf
            w = scores.gather(1, choice.topk(k, 1).indices)
            return None, w * c["scale"] / (w.sum(1, keepdim=True) if c["renorm"] else 1)
        g = s["dweights"].double() * c["scale"]
        ids = s["ids"].long()
        row = torch.arange(t, device="cuda")[:, None].expand_as(ids)
        leaf = logits.requires_grad_(True)
        p = torch.sigmoid(leaf) if c["score"] == "sigmoid" else torch.softmax(leaf, 1)
        w = p[row, ids]
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad((w * g).sum(), leaf)[0].detach()
    if kind == "dispatch":
        # pairs by expert, then by token
        pair = torch.arange(t * k, device="cuda")
        order = torch.sort(s["ids"].reshape(-1).long() * (t * k) + pair).indices
        return None, None, s["x"].double()[order // k]
    slots, w = s["slots"].long(), s["weights"].double()
    if kind == "combine":
        mix = torch.zeros(t, c["hidden"], dtype=torch.float64, device="cuda")
        for j in range(k):
            mix.addcmul_(s["rows"][slots[:, j]].double(), w[:, j:j + 1])
        return mix
    dy, drows, dw = s["dy"].double(), torch.empty(t * k, c["hidden"], dtype=torch.float64, device="cuda"), []
    for j in range(k):
        drows[slots[:, j]] = w[:, j:j + 1] * dy
        dw.append(torch.einsum("th,th->t", dy, s["rows"][slots[:, j]].double()))
    return drows, torch.stack(dw, 1)
