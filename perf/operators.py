"""The block-scaled FP8 products and the expert router: what is measured of them.

Every case is one pass as a program makes it: a quantizer call, a linear layer from BF16 activations to BF16
outputs, an expert projection from a router's choices to the packed rows of every expert, or a router's step
(packing, balance loss and its gradient).  With ``own`` false the same results come from elementary torch
operations in 32 bits.

FP8 format: E4M3 codes; one FP32 scale for each 128 consecutive K-values of an activation row, and for each
128 x 128 block of a weight [N, K]; s = amax / 448 (1 for a block of zeros), code = E4M3(x / s) to nearest even.
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # the largest E4M3 value


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's activations: 64 tokens of the o_proj input
        {"name": "quant act 64x8192", "kind": "quant_act", "m": 64, "k": 8192},
        # a prefill chunk, odd row count
        {"name": "quant act 8191x8192", "kind": "quant_act", "m": 8191, "k": 8192},
        # checkpoint conversion of the o_proj weight
        {"name": "quant weight 7168x8192", "kind": "quant_weight", "n": 7168, "k": 8192},
        # a single token through the layer: latency and the weight stream
        {"name": "linear 1x7168x8192", "kind": "linear", "m": 1, "n": 7168, "k": 8192},
        # batched decode, 8 requests x 8 draft positions
        {"name": "linear 64x7168x8192", "kind": "linear", "m": 64, "n": 7168, "k": 8192},
        # a ragged chunk between decode and prefill on a narrow odd projection
        {"name": "linear 777x1100x2176", "kind": "linear", "m": 777, "n": 1100, "k": 2176},
        # prefill of 8 prompts of 1024 tokens
        {"name": "linear 8192x7168x8192", "kind": "linear", "m": 8192, "n": 7168, "k": 8192},
        # experts' up projection in decode: 64 tokens x top-8 over 32 experts
        {"name": "experts 64x8 of 32", "kind": "experts", "t": 64, "top": 8, "e": 32, "n": 2048, "k": 7168},
        # the same projection over a prefill chunk
        {"name": "experts 2048x8 of 32", "kind": "experts", "t": 2048, "top": 8, "e": 32, "n": 2048, "k": 7168},
        # a router's step on a decode-sized batch: launches only
        {"name": "router 64x32 top 8", "kind": "router", "t": 64, "e": 32, "top": 8, "half": False, "pad": False},
        # odd sizes, BF16 logits, padded tokens
        {"name": "router 4099x160 top 6", "kind": "router", "t": 4099, "e": 160, "top": 6, "half": True, "pad": True},
        # a training micro-batch
        {"name": "router 16384x256 top 8", "kind": "router", "t": 16384, "e": 256, "top": 8, "half": False, "pad": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["quant_act", "quant_weight", "linear", "linear", "linear", "experts", "experts", "router", "router"])
    if kind == "quant_act":
        return {"kind": kind, "m": _spread(rng, 1, 8192), "k": BLOCK * _spread(rng, 4, 64)}
    if kind == "quant_weight":
        return {"kind": kind, "n": _spread(rng, 100, 8192), "k": BLOCK * _spread(rng, 4, 64)}
    if kind == "linear":
        return {"kind": kind, "m": _spread(rng, 1, 8192), "n": _spread(rng, 256, 7168), "k": BLOCK * _spread(rng, 4, 64)}
    if kind == "experts":
        e = _spread(rng, 8, 64)
        return {"kind": kind, "t": _spread(rng, 1, 1024), "top": rng.randint(1, 8), "e": e, "n": _spread(rng, 256, 2048),
                "k": BLOCK * _spread(rng, 8, 40)}
    e = _spread(rng, 8, 256)
    return {"kind": kind, "t": _spread(rng, 1, 16384), "e": e, "top": rng.randint(1, 8), "half": rng.random() < 0.5,
            "pad": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _activations(gen, m, k):
    """Normal activations, tokens of different size, with 1% of the columns 30 times as large."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=gen, device="cuda"))
    wide = torch.rand((1, k), generator=gen, device="cuda") < 0.01
    return torch.where(wide, x * 30, x).to(torch.bfloat16)


def _weight(gen, n, k):
    """Normal weights, output channels of different size."""
    return torch.randn((n, k), generator=gen, device="cuda") * torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda")) * 0.02


def _codes_of_weight(gen, n, k):
    """A stored weight: uint8 E4M3 codes and block scales."""
    q, s = _plain_quant_weight(_weight(gen, n, k))
    return q.view(torch.uint8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "quant_act":
        return {"kind": kind, "x": _activations(gen, case["m"], case["k"])}
    if kind == "quant_weight":
        return {"kind": kind, "w": _weight(gen, case["n"], case["k"])}
    if kind == "linear":
        qw, sw = _codes_of_weight(gen, case["n"], case["k"])
        return {"kind": kind, "x": _activations(gen, case["m"], case["k"]), "qw": qw, "sw": sw}
    t, e, top = case["t"], case["e"], min(case["top"], case["e"])
    # some experts are preferred, so that groups differ in size
    logits = 1.5 * torch.randn((t, e), generator=gen, device="cuda") + 0.5 * torch.randn((1, e), generator=gen, device="cuda")
    if kind == "experts":
        ids = logits.topk(top, dim=1).indices
        stored = [_codes_of_weight(gen, case["n"], case["k"]) for _ in range(e)]
        return {"kind": kind, "x": _activations(gen, t, case["k"]), "ids": ids, "qw": torch.stack([q for q, _ in stored]),
                "sw": torch.stack([s for _, s in stored]), "most": int(torch.bincount(ids.reshape(-1), minlength=e).max())}
    logits = logits.to(torch.bfloat16 if case["half"] else torch.float32)
    ids = logits.topk(top, dim=1).indices
    mask = None
    if case["pad"]:  # padded tokens: no expert, no share in the loss
        mask = torch.rand((t,), generator=gen, device="cuda") < 0.85
        ids = torch.where(mask[:, None], ids, -1)
    return {"kind": kind, "logits": logits, "ids": ids, "e": e, "coef": 0.01, "mask": mask,
            "grad": torch.rand((1,), generator=gen, device="cuda") + 0.5}


# ---------------------------------------------------------------- plain forms
def _scale(a):
    # by a tensor: torch turns a division by a number into a product with its rounded inverse, and a scale that is
    # off by its last bit moves codes that lie on a border
    return torch.where(a == 0, 1.0, a / torch.full_like(a, TOP))


def _plain_quant_act(x):
    m, k = x.shape
    v = x.float().view(m, k // BLOCK, BLOCK)
    a = v.abs().amax(dim=2)
    s = _scale(a)
    return (v / s[..., None]).view(m, k).to(torch.float8_e4m3fn), s


def _plain_quant_weight(w):
    n, k = w.shape
    nb = -(-n // BLOCK)
    v = torch.nn.functional.pad(w, (0, 0, 0, nb * BLOCK - n)).view(nb, BLOCK, k // BLOCK, BLOCK)
    a = v.abs().amax(dim=(1, 3))
    s = _scale(a)
    return (v / s[:, None, :, None]).view(nb * BLOCK, k)[:n].to(torch.float8_e4m3fn), s


def _values_of_act(q, s):
    return (q.view(torch.float8_e4m3fn).float().view(*s.shape, BLOCK) * s[..., None]).view(q.shape)


def _values_of_weight(q, s):
    """E4M3 codes [..., N, K] and block scales [..., N / 128 rounded up, K / 128] -> FP32 values."""
    rows = s.repeat_interleave(BLOCK, dim=-2)[..., : q.shape[-2], :]
    v = q.view(torch.float8_e4m3fn).float().view(*q.shape[:-1], q.shape[-1] // BLOCK, BLOCK)
    return (v * rows[..., None]).view(q.shape)


def _plain_linear(x, qw, sw):
    return (_values_of_act(*_plain_quant_act(x)) @ _values_of_weight(qw, sw).t()).to(torch.bfloat16)


def _plain_route(ids, e):
    """counts, offsets, the token of every packed row (-1 behind the last) and the packed row of every choice."""
    t, top = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < e)
    counts = (flat[None, :] == torch.arange(e, device=ids.device)[:, None]).sum(dim=1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.where(ok, flat, e).sort(stable=True).indices
    packed = torch.arange(t * top, device=ids.device)
    rows = torch.where(packed < offsets[-1], order // top, -1)
    slots = torch.empty_like(packed)
    slots[order] = packed
    slots = torch.where(ok, slots, -1).view(t, top)
    return counts.int(), offsets.int(), rows.int(), slots.int()


def _plain_experts(x, ids, qw, sw, most):
    e, n, k = qw.shape
    counts, offsets, rows, slots = _plain_route(ids, e)
    v = _values_of_act(*_plain_quant_act(x))
    place = offsets[:-1, None].long() + torch.arange(most, device=x.device)  # packed rows, expert by expert, padded
    held = torch.arange(most, device=x.device) < counts[:, None]
    place = torch.where(held, place, 0)
    a = torch.where(held[..., None], v[rows.long()[place].clamp(min=0)], 0.0)
    y = torch.bmm(_values_of_weight(qw, sw), a.transpose(1, 2).contiguous()).transpose(1, 2)  # [e, most, n]
    return y[held].to(torch.bfloat16)


def _plain_balance(logits, counts, coef, mask, grad):
    t, e = logits.shape
    p = torch.softmax(logits.float(), dim=1)
    live = torch.ones(t, device=logits.device) if mask is None else mask.float()
    f = counts.float() / counts.sum().clamp(min=1)
    w = coef * e * f / live.sum().clamp(min=1)
    per = (p * w).sum(dim=1)
    loss = (per * live).sum()
    d = grad * live[:, None] * p * (w - per[:, None])
    return loss.view(1), d.to(logits.dtype)


# ---------------------------------------------------------------- one pass
def run(state):
    kind = state["kind"]
    if own:
        from block_scaled_precision_act_amd import mxgemm
        if kind == "quant_act":
            q, s = mxgemm.quant_act_b128(state["x"])
            return {"q": q.view(torch.float8_e4m3fn), "s": s}
        if kind == "quant_weight":
            q, s = mxgemm.quant_weight_b128(state["w"])
            return {"q": q.view(torch.float8_e4m3fn), "s": s}
        if kind == "linear":
            return {"y": mxgemm.linear_a8w8_b128(state["x"], state["qw"], state["sw"])}
        if kind == "experts":
            _, offsets, rows, _ = mxgemm.moe_route(state["ids"], state["qw"].shape[0])
            qa, sa = mxgemm.quant_act_b128(state["x"])
            return {"y": mxgemm.gemm_a8w8_b128_grouped(qa, sa, state["qw"], state["sw"], offsets, rows=rows)}
        counts, offsets, rows, slots = mxgemm.moe_route(state["ids"], state["e"])
        loss, w = mxgemm.moe_balance_loss(state["logits"], counts, state["coef"], mask=state["mask"])
        d = mxgemm.moe_balance_loss_grad(state["logits"], w, state["grad"], mask=state["mask"])
        return {"counts": counts, "offsets": offsets, "rows": rows, "slots": slots, "loss": loss, "dlogits": d}
    if kind == "quant_act":
        q, s = _plain_quant_act(state["x"])
        return {"q": q, "s": s}
    if kind == "quant_weight":
        q, s = _plain_quant_weight(state["w"])
        return {"q": q, "s": s}
    if kind == "linear":
        return {"y": _plain_linear(state["x"], state["qw"], state["sw"])}
    if kind == "experts":
        return {"y": _plain_experts(state["x"], state["ids"], state["qw"], state["sw"], state["most"])}
    counts, offsets, rows, slots = _plain_route(state["ids"], state["e"])
    loss, d = _plain_balance(state["logits"], counts, state["coef"], state["mask"], state["grad"])
    return {"counts": counts, "offsets": offsets, "rows": rows, "slots": slots, "loss": loss, "dlogits": d}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    if kind == "quant_act":
        m, k = case["m"], case["k"]
        return {"bytes": 3 * m * k + 4 * m * (k // BLOCK), "flops": 2 * m * k}
    if kind == "quant_weight":
        n, k = case["n"], case["k"]
        return {"bytes": 5 * n * k + 4 * -(-n // BLOCK) * (k // BLOCK), "flops": 2 * n * k}
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k + 4 * -(-n // BLOCK) * (k // BLOCK) + 2 * m * n, "flops": 2 * m * n * k}
    t, e = case["t"], case["e"]
    top = min(case["top"], e)
    if kind == "experts":
        n, k = case["n"], case["k"]
        hit = e * (1 - (1 - top / e) ** t)  # experts that some token chose, about
        return {"bytes": 2 * t * k + 8 * t * top + hit * (n * k + 4 * -(-n // BLOCK) * (k // BLOCK)) + 2 * t * top * n,
                "flops": 2 * t * top * n * k}
    size = 2 if case["half"] else 4
    return {"bytes": 2 * size * t * e + 8 * t * top + 8 * t * top + 8 * e + (t if case["pad"] else 0), "flops": 12 * t * e}


# ---------------------------------------------------------------- the definition in 64 bits
def _e4m3(v):
    """FP64 values rounded onto the E4M3 grid, ties to even."""
    exponent = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_codes(v, a):
    """v [..., values] and its blocks' largest magnitudes, broadcastable: code values and scales, the scale and the
    quotient rounded to FP32 as the format has it."""
    s = torch.where(a == 0, torch.ones_like(a), (a / torch.full_like(a, TOP)).float().double())
    return _e4m3((v / s).float().double()), s


def _exact_act(x):
    v = x.double().reshape(x.shape[0], -1, BLOCK)
    c, s = _exact_codes(v, v.abs().amax(dim=2, keepdim=True))
    return c, s


def exact(case, seed):
    state = prepare(case, seed)
    kind = state["kind"]
    if kind == "quant_act":
        c, s = _exact_act(state["x"])
        return {"q": c.reshape(state["x"].shape), "s": s[..., 0]}
    if kind == "quant_weight":
        w = state["w"].double()
        q, s = torch.empty_like(w), []
        for r in range(0, w.shape[0], BLOCK):
            v = w[r:r + BLOCK].reshape(-1, w.shape[1] // BLOCK, BLOCK)
            c, scale = _exact_codes(v, v.abs().amax(dim=(0, 2), keepdim=True))
            q[r:r + BLOCK] = c.reshape(v.shape[0], -1)
            s.append(scale.reshape(1, -1))
        return {"q": q, "s": torch.cat(s)}
    if kind in ("linear", "experts"):
        c, s = _exact_act(state["x"])
        a = (c * s).reshape(state["x"].shape)

        def weight(q, scale):
            up = torch.ones((BLOCK, BLOCK), dtype=torch.float64, device=q.device)
            return q.view(torch.float8_e4m3fn).double() * torch.kron(scale.double(), up)[: q.shape[0]]
        if kind == "linear":
            return {"y": a @ weight(state["qw"], state["sw"]).t()}
        parts = []
        for e in range(state["qw"].shape[0]):
            token = (state["ids"] == e).nonzero()[:, 0]  # in the order of tokens; a token chooses an expert once
            parts.append(a[token] @ weight(state["qw"][e], state["sw"][e]).t())
        return {"y": torch.cat(parts)}
    logits, ids, e = state["logits"].double(), state["ids"], state["e"]
    t, top = ids.shape
    live = torch.ones(t, dtype=torch.bool, device=ids.device) if state["mask"] is None else state["mask"]
    rows = torch.full((t * top,), -1, dtype=torch.int64, device=ids.device)
    slots = torch.full((t, top), -1, dtype=torch.int64, device=ids.device)
    counts, at = [], 0
    for x in range(e):
        where = (ids == x).nonzero()
        rows[at:at + len(where)] = where[:, 0]
        slots[where[:, 0], where[:, 1]] = torch.arange(at, at + len(where), device=ids.device)
        counts.append(len(where))
        at += len(where)
    n = torch.tensor(counts, device=ids.device)
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    z = (logits - logits.logsumexp(dim=1, keepdim=True)).exp()[live]
    f = n.double() / max(at, 1)
    tokens = max(int(live.sum()), 1)
    loss = state["coef"] * e * (f * (z.sum(dim=0) / tokens)).sum()
    d = torch.zeros_like(logits)
    upstream = state["grad"].double() * state["coef"] * e / tokens
    d[live] = upstream * (z * f - z * (z @ f)[:, None])  # the softmax's Jacobian applied to f
    return {"counts": n.int(), "offsets": offsets.int(), "rows": rows.int(), "slots": slots.int(), "loss": loss.view(1), "dlogits": d}
