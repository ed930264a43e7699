"""The operators of a feed-forward unit, as a training or serving step runs them.

An FSDP unit's parameters arrive in per-parameter bf16 storage, its feed-forward
block computes from them, and its gradients leave through the reduce-scatter.
Four kinds of call stand between the two:

  forward   h = act(x Wg^T) * (x Wu^T); with a checkpoint the pre-activations
            are kept in 8 bits (e4m3, a power-of-two scale for each 1 x 128)
  backward  dx, dWg, dWu from dh; the pre-activations recomputed, or read from
            the 8-bit checkpoint
  store / restore   bf16 to 8-bit blocks and back (1 x 128 for activations,
            128 x 128 for weights)
  matmul    out = A B^T from 8-bit blocks, A with a scale for each 1 x 128 and
            B with one for each 128 x 128

`run` computes them in plain torch operations in 32 bits, or, with `own`, by the
framework's kernels.
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


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one generated token through an 8B-shaped feed-forward block
        dict(name="forward_token_8b", kind="forward", m=1, k=4096, f=14336, act="silu", keep=False),
        # a ragged handful of tokens routed to one 768-wide expert, training
        dict(name="forward_expert_37", kind="forward", m=37, k=2048, f=768, act="silu", keep=True),
        # a 2048-token prompt through the 8B-shaped block, tanh-GELU gate
        dict(name="forward_8b_2048", kind="forward", m=2048, k=4096, f=14336, act="gelu", keep=False),
        # a training step's tokens through the 70B-shaped block, kept in 8 bits
        dict(name="forward_70b_4093", kind="forward", m=4093, k=8192, f=28672, act="silu", keep=True),
        # the tiny block's backward pass with 250 tokens, recomputed
        dict(name="backward_tiny_250", kind="backward", m=250, k=256, f=704, act="silu", keep=False),
        # one expert's backward pass from its 8-bit checkpoint, odd token count
        dict(name="backward_expert_1021", kind="backward", m=1021, k=2048, f=768, act="silu", keep=True),
        # the 8B-shaped block's backward pass, recomputed
        dict(name="backward_8b_2048", kind="backward", m=2048, k=4096, f=14336, act="gelu", keep=False),
        # the 70B-shaped block's backward pass from its 8-bit checkpoint
        dict(name="backward_70b_4096", kind="backward", m=4096, k=8192, f=28672, act="silu", keep=True),
        # a 70B-shaped weight to 128 x 128 blocks, after its placement
        dict(name="store_weight_70b", kind="store", rows=28672, cols=8192, block_rows=128),
        # a ragged batch of activations back from its checkpoint
        dict(name="restore_4093", kind="restore", rows=4093, cols=8192, block_rows=1),
        # one token through the 70B-shaped down projection in 8 bits
        dict(name="matmul_token_70b", kind="matmul", m=1, n=8192, k=28672),
        # a prompt's tokens through the 70B-shaped down projection in 8 bits
        dict(name="matmul_70b_4093", kind="matmul", m=4093, n=8192, k=28672),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "backward", "store", "restore", "matmul", "matmul"])
    if kind in ("store", "restore"):
        # codes are stored whole, so any width: every other one is odd
        cols = _log(rng, 64, 28672)
        cols = cols | 1 if rng.random() < 0.5 else (cols + 7) // 8 * 8
        return dict(kind=kind, rows=_log(rng, 1, 8192), cols=cols, block_rows=rng.choice([1, 128]))
    m = _log(rng, 1, 4096)
    k = (_log(rng, 128, 8192) + 15) // 16 * 16
    f = (_log(rng, 128, 28672) + 15) // 16 * 16
    if kind == "matmul":
        return dict(kind=kind, m=m, n=k, k=f)
    return dict(kind=kind, m=m, k=k, f=f, act=rng.choice(["silu", "gelu"]), keep=rng.random() < 0.5)


def work(case):
    c = case
    if c["kind"] in ("store", "restore"):
        r, n, b = c["rows"], c["cols"], c["block_rows"]
        return {"bytes": 3 * r * n + 4 * -(-r // b) * -(-n // 128), "flops": 2 * r * n}
    m, k = c["m"], c["k"]
    if c["kind"] == "matmul":
        n, kb = c["n"], -(-k // 128)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // 128)) + 2 * m * n, "flops": 2 * m * n * k}
    f = c["f"]
    eight = 2 * m * f + 8 * m * -(-f // 128)  # codes and scales of the two pre-activations
    if c["kind"] == "forward":
        # with a checkpoint its values come back too, as bf16
        return {"bytes": 2 * (m * k + 2 * f * k + m * f) + (2 * eight + 4 * m * f if c["keep"] else 0), "flops": 4 * m * k * f}
    x8 = m * k + 4 * m * -(-k // 128)
    return {"bytes": 2 * m * f + (eight + x8 if c["keep"] else 2 * m * k) + 4 * f * k + 2 * m * k + 4 * f * k,
            "flops": (8 if c["keep"] else 12) * m * k * f}


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) * scale).to(torch.bfloat16)


def _acts(g, rows, cols):
    """Activations as they come: every row with its own size, one channel in 64 an outlier."""
    x = _randn(g, rows, cols)
    x *= torch.exp2(torch.randint(-2, 3, (rows, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    x[:, ::64] *= 16.0
    return x


def _to_blocks(v, block_rows):
    """(e4m3 codes, float32 scales) of a float32 matrix, one scale for each block_rows x 128.

    The scale is the smallest power of two (at least 2^-126) that brings the
    block's largest finite value to 448 or below, 1 for a block of zeros."""
    r, c = v.shape
    nr, nc = -(-r // block_rows), -(-c // 128)
    p = torch.zeros(nr * block_rows, nc * 128, dtype=torch.float32, device=v.device)
    p[:r, :c] = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    amax = p.view(nr, block_rows, nc, 128).abs().amax(dim=(1, 3))
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(min=-126)
    scales = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    each = scales.repeat_interleave(block_rows, 0)[:r].repeat_interleave(128, 1)[:, :c]
    return (v / each).to(torch.float8_e4m3fn), scales


def _from_blocks(codes, scales, block_rows):
    r, c = codes.shape
    return codes.float() * scales.repeat_interleave(block_rows, 0)[:r].repeat_interleave(128, 1)[:, :c]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["kind"] in ("store", "restore"):
        r, n, b = c["rows"], c["cols"], c["block_rows"]
        src = _acts(g, r, n) if b == 1 else _randn(g, r, n, scale=0.02)
        if c["kind"] == "store":
            s.update(src=src, codes=new(r, n, dtype=torch.float8_e4m3fn), scales=new(-(-r // b), -(-n // 128), dtype=torch.float32))
        else:
            codes, scales = _to_blocks(src.float(), b)
            s.update(codes=codes, scales=scales, dst=new(r, n))
        return s
    m, k = c["m"], c["k"]
    if c["kind"] == "matmul":
        n = c["n"]
        s["a"], s["sa"] = _to_blocks(_acts(g, m, k).float(), 1)
        s["b"], s["sb"] = _to_blocks(_randn(g, n, k, scale=k ** -0.5).float(), 128)
        s["out"] = new(m, n)
        return s
    f = c["f"]
    x = _acts(g, m, k)
    s.update(wg=_randn(g, f, k, scale=0.5 * k ** -0.5), wu=_randn(g, f, k, scale=0.5 * k ** -0.5))
    if c["kind"] == "forward":
        s.update(x=x, h=new(m, f))
        if c["keep"]:  # gate rows, then up rows
            s.update(codes=new(2 * m, f, dtype=torch.float8_e4m3fn), scales=new(2 * m, -(-f // 128), dtype=torch.float32), values=new(2 * m, f))
        return s
    s.update(dh=_randn(g, m, f, scale=1.0 / 64), dx=new(m, k), dwg=new(f, k), dwu=new(f, k))
    if c["keep"]:
        s["x8"], s["sx"] = _to_blocks(x.float(), 1)
        s["codes"], s["scales"] = _to_blocks(torch.randn(2 * m, f, generator=g, device="cuda"), 1)
    else:
        s["x"] = x
    return s


# ---------------------------------------------------------------- one pass

def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * b * g * g)


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "store":
        return _to_blocks(s["src"].float(), c["block_rows"])
    if kind == "restore":
        return _from_blocks(s["codes"], s["scales"], c["block_rows"]).bfloat16()
    if kind == "matmul":
        return (_from_blocks(s["a"], s["sa"], 1) @ _from_blocks(s["b"], s["sb"], 128).T).bfloat16()
    m, wg, wu = c["m"], s["wg"].float(), s["wu"].float()
    if kind == "forward":
        x = s["x"].float()
        g, u = x @ wg.T, x @ wu.T
        h = (_act(g, c["act"])[0] * u).bfloat16()
        if not c["keep"]:
            return h
        return h, _from_blocks(*_to_blocks(torch.cat([g, u]), 1), 1).bfloat16()
    if c["keep"]:
        x, gu = _from_blocks(s["x8"], s["sx"], 1), _from_blocks(s["codes"], s["scales"], 1)
        g, u = gu[:m], gu[m:]
    else:
        x = s["x"].float()
        g, u = x @ wg.T, x @ wu.T
    dh = s["dh"].float()
    a, da = _act(g, c["act"])
    du, dg = dh * a, dh * u * da
    return (dg @ wg + du @ wu).bfloat16(), (dg.T @ x).bfloat16(), (du.T @ x).bfloat16()


def _run_own(s):
    import layout_aware_collectives_gb300 as tide

    c, t, stream = s["case"], _compute(), torch.cuda.current_stream()
    kind = c["kind"]
    if kind == "store":
        t.fp8_store(c["rows"], c["cols"], s["src"], s["codes"], s["scales"], block_rows=c["block_rows"], stream=stream)
        return s["codes"], s["scales"]
    if kind == "restore":
        t.fp8_restore(c["rows"], c["cols"], s["codes"], s["scales"], s["dst"], block_rows=c["block_rows"], stream=stream)
        return s["dst"]
    if kind == "matmul":
        t.fp8_matmul(c["m"], c["n"], c["k"], s["a"], s["sa"], s["b"], s["sb"], s["out"], stream=stream)
        return s["out"]
    m, k, f = c["m"], c["k"], c["f"]
    keep = None
    if c["keep"]:
        if "checkpoint" not in s:
            s["checkpoint"] = tide.GatedCheckpoint(s["codes"][:m], s["scales"][:m], s["codes"][m:], s["scales"][m:], s.get("x8"), s.get("sx"))
        keep = s["checkpoint"]
    if kind == "forward":
        t.gated_forward(m, k, f, s["x"], s["wg"], s["wu"], s["h"], activation=c["act"], checkpoint=keep, stream=stream)
        if keep is None:
            return s["h"]
        t.fp8_restore(2 * m, f, s["codes"], s["scales"], s["values"], stream=stream)
        return s["h"], s["values"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(tide.gated_workspace_bytes(m, k, f), dtype=torch.uint8, device="cuda")
    t.gated_backward(m, k, f, s["dh"], s.get("x"), s["wg"], s["wu"], s["dx"], s["dwg"], s["dwu"], s["workspace"],
                     activation=c["act"], checkpoint=keep, stream=stream)
    return s["dx"], s["dwg"], s["dwu"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- in 64 bits

def _widen(codes, scales, block_rows):
    """The blocks' values in 64 bits: each element's scale by its indexes."""
    i = torch.arange(codes.shape[0], device=codes.device) // block_rows
    j = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.double() * scales.double()[i][:, j]


def exact(case, seed):
    """What run() returns, in 64 bits.  What is held in 8 bits is given as the
    value before that rounding, so both sides show the format's own error."""
    s, c = prepare(case, seed), case
    kind = c["kind"]
    if kind == "store":
        v = s["src"].double()
        r, n = v.shape
        b, nc = c["block_rows"], -(-n // 128)
        i = torch.arange(r, device="cuda") // b
        j = torch.arange(n, device="cuda") // 128
        top = torch.zeros(-(-r // b) * nc, dtype=torch.float64, device="cuda")
        top = top.scatter_reduce(0, (i[:, None] * nc + j).reshape(-1), v.abs().reshape(-1), "amax").view(-1, nc)
        scale = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448)))
        return v / scale[i][:, j], scale
    if kind == "restore":
        return _widen(s["codes"], s["scales"], c["block_rows"])
    if kind == "matmul":
        return _widen(s["a"], s["sa"], 1) @ _widen(s["b"], s["sb"], 128).T
    m = c["m"]
    wg, wu = s["wg"].double(), s["wu"].double()
    if c["kind"] == "backward" and c["keep"]:
        x = _widen(s["x8"], s["sx"], 1)
        g, u = _widen(s["codes"], s["scales"], 1).split(m)
    else:
        x = s["x"].double()
        g, u = x @ wg.T, x @ wu.T
    if c["act"] == "silu":
        a = g * torch.sigmoid(g)
        slope = torch.sigmoid(g) + a * (1 - torch.sigmoid(g))
    else:
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        # 0.5 (1 + tanh z) = sigmoid(2 z)
        a = g * torch.sigmoid(2 * z)
        dz = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
        slope = torch.sigmoid(2 * z) + 2 * g * torch.sigmoid(2 * z) * torch.sigmoid(-2 * z) * dz
    if kind == "forward":
        return (a * u, torch.cat([g, u])) if c["keep"] else a * u
    dh = s["dh"].double()
    dg, du = dh * u * slope, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x
