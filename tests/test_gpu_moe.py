"""GPU parity of the expert routing: packing exactly, the balance loss and its gradient against float64, and the whole
path from a router's logits to the experts' products."""
import numpy as np
import pytest

import b128
from block_scaled_precision_act_amd import synth
from parity import bf16_dev, bf16_host, to_dev

pytestmark = pytest.mark.gpu


def _route(ids, e):
    t, top = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < e)
    key = np.where(ok, flat, e)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=e + 1)[:e]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    rows = np.full(t * top, -1)
    rows[:offsets[-1]] = order[:offsets[-1]] // max(top, 1)
    slots = np.full(t * top, -1)
    slots[order[:offsets[-1]]] = np.arange(offsets[-1])
    return counts, offsets, rows, slots.reshape(t, top)


@pytest.mark.parametrize("t,top,e", [
    (1, 1, 1), (1, 8, 8), (64, 8, 32), (63, 3, 7), (1000, 2, 1000), (8192, 1, 1024), (1025, 8, 3), (8191, 1, 5), (4097, 2, 64),
    (1000, 9, 160), (20000, 8, 256), (65537, 1, 2), (300, 100, 1024), (65536, 1, 1024), (2048, 1, 40), (2049, 1, 40), (40000, 3, 1000),
])
@pytest.mark.parametrize("wide", [False, True])
def test_route_exact(mx, t, top, e, wide):
    import torch
    rng = np.random.default_rng(t + e)
    ids = rng.integers(-2, e + 2, (t, top))
    ids = np.where(rng.random((t, 1)) < 0.1, -1, ids)  # padded tokens
    if wide:
        ids[rng.random(ids.shape) < 0.02] = (1 << 40) + 1  # not 1 in the low half
    got = mx.moe_route(to_dev(ids.astype(np.int64 if wide else np.int32)), e)
    for name, g, w in zip(("counts", "offsets", "rows", "slots"), got, _route(ids, e)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), name


# from 32768 counts of chunks on: more chunks than threads for an expert, fewer, a last chunk of one, the most choices
@pytest.mark.parametrize("t,top,e", [(70000, 8, 160), (69633, 1, 1000), (65536, 8, 129), (1 << 21, 8, 256), (1 << 24, 1, 5)])
def test_route_many_choices(mx, t, top, e):
    rng = np.random.default_rng(t + e)
    ids = rng.integers(-2, e + 2, (t, top)).astype(np.int32)
    got = mx.moe_route(to_dev(ids), e)
    for name, g, w in zip(("counts", "offsets", "rows", "slots"), got, _route(ids, e)):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("t,top,e", [(0, 4, 6), (5, 0, 6), (300, 2, 9), (9000, 2, 9)])
def test_route_without_choices(mx, t, top, e):
    ids = np.full((t, top), -1, np.int64)
    counts, offsets, rows, slots = (g.cpu().numpy() for g in mx.moe_route(to_dev(ids), e))
    assert not counts.any() and not offsets.any() and (rows == -1).all() and (slots == -1).all() and slots.shape == (t, top)


@pytest.mark.parametrize("t", [700, 30000, 70000])
def test_route_one_expert_takes_all(mx, t):
    ids = np.full((t, 1), 17, np.int32)
    counts, offsets, rows, slots = (g.cpu().numpy() for g in mx.moe_route(to_dev(ids), 40))
    assert counts[17] == t and np.array_equal(rows, np.arange(t)) and np.array_equal(slots[:, 0], np.arange(t))
    assert (offsets[:18] == 0).all() and (offsets[18:] == t).all()


# ---------------------------------------------------------------- balance loss
# Relative error of a probability: the exponent's argument is off by 2^-24 of its size (up to 40 here), the exponential by
# 2^-23, the sum of E <= 1024 positive values by at most 22 roundings, and the quotient by two: (40 + 2 + 22 + 2) 2^-24.
# A weighted sum of them adds at most 22 more, and the weights one each: below 90 * 2^-24.
EPS = 90 * 2.0 ** -24


def _balance(logits, counts, coef, mask, grad):
    """Loss, weights, gradient and the gradient's error scale in float64."""
    t, e = logits.shape
    z = logits.astype(np.float64)
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.exp(z - np.where(np.isneginf(top), 0, top))
        s = p.sum(1, keepdims=True)
        p = p / np.where(s == 0, 1, s)
    live = np.ones(t, bool) if mask is None else mask.astype(bool)
    n, total = live.sum(), counts.sum()
    w = coef * e * counts / max(total, 1) / max(n, 1) if n and total else np.zeros(e)
    p = np.where(live[:, None], p, 0)  # padded rows may hold anything
    per = p @ w
    d = grad * p * (w - per[:, None])
    return per.sum(), w, d, abs(grad) * p * (w + 2 * per[:, None])


def _bf16(a):
    return synth.f64_to_bf16_bits(np.ascontiguousarray(a.reshape(-1), np.float64)).reshape(a.shape)


@pytest.mark.parametrize("t,e", [(1, 1), (1, 7), (64, 32), (33, 8), (100, 16), (77, 60), (1000, 128), (513, 160), (4099, 256),
                                 (300, 500), (129, 1024), (9001, 12)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("padded", [False, True])
def test_balance_loss_and_gradient(mx, t, e, half, padded):
    import torch
    rng = np.random.default_rng(t + e)
    logits = rng.normal(0, 3, (t, e))
    logits[rng.random((t, e)) < 0.05] = -np.inf  # experts that are closed
    logits[:, 0] = np.where(np.isneginf(logits).all(1), 0, logits[:, 0])
    if t > 20:
        logits[11] = -np.inf  # nothing left
    mask = rng.random(t) < 0.8 if padded else None
    if padded and t > 20:
        logits[~mask] = np.nan
    counts = rng.integers(0, 50, e).astype(np.int32)
    if half:
        ld = bf16_dev(_bf16(np.nan_to_num(logits, nan=0, neginf=0)))
        ld[torch.from_numpy(np.isneginf(logits)).cuda()] = float("-inf")
        ld[torch.from_numpy(np.isnan(logits)).cuda()] = float("nan")
        logits = bf16_host(ld)
    else:
        ld = to_dev(logits.astype(np.float32))
        logits = logits.astype(np.float32)
    coef, grad = 0.02, -1.7
    loss, w, d, scale = _balance(logits, counts, coef, mask, np.float32(grad).astype(np.float64))
    md = None if mask is None else to_dev(mask)
    gl, gw = mx.moe_balance_loss(ld, to_dev(counts), coef, mask=md)
    gd = mx.moe_balance_loss_grad(ld, gw, torch.tensor([grad], device="cuda"), mask=md)
    # the coefficient is passed in FP32: half a step more
    assert abs(float(gl) - loss) <= (EPS + 2.0 ** -24) * loss + 1e-38
    assert np.all(np.abs(gw.cpu().numpy() - w) <= 2.0 ** -23 * w)
    gh = bf16_host(gd) if half else gd.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(gh - d) <= EPS * scale + (2.0 ** -8 if half else 2.0 ** -23) * np.abs(d) + 1e-38)
    if mask is not None:
        assert not gh[~mask].any()


# rows that are no multiple of their loads, and rows that start between them
@pytest.mark.parametrize("t,e,shift", [(50, 65, 0), (50, 131, 0), (3, 255, 0), (40, 257, 0), (20, 1023, 0), (40, 70, 1),
                                       (50, 160, 1), (50, 160, 2), (40, 512, 3), (20, 1000, 1), (600, 256, 1)])
@pytest.mark.parametrize("half", [False, True])
def test_balance_rows_of_any_start(mx, t, e, shift, half):
    import torch
    rng = np.random.default_rng(t * e + shift)
    logits = rng.normal(0, 3, (t, e))
    mask = rng.random(t) < 0.7
    mask[0] = True
    logits[~mask] = np.nan
    buf = torch.zeros(t * e + shift, dtype=torch.bfloat16 if half else torch.float32, device="cuda")
    ld = buf[shift:].view(t, e)
    ld.copy_(torch.from_numpy(logits))
    logits = bf16_host(ld) if half else ld.cpu().numpy()
    counts = rng.integers(0, 50, e).astype(np.int32)
    coef, grad = 0.02, -1.7
    loss, w, d, scale = _balance(logits, counts, coef, mask, np.float32(grad).astype(np.float64))
    gl, gw = mx.moe_balance_loss(ld, to_dev(counts), coef, mask=to_dev(mask))
    out = torch.full((t * e + shift + 8,), 7.0, dtype=ld.dtype, device="cuda")
    mx.moe_balance_loss_grad(ld, gw, torch.tensor([grad], device="cuda"), mask=to_dev(mask), dlogits=out[shift:shift + t * e].view(t, e))
    assert (out[:shift] == 7).all() and (out[shift + t * e:] == 7).all()
    gd = out[shift:shift + t * e].view(t, e)
    gh = bf16_host(gd) if half else gd.cpu().numpy().astype(np.float64)
    assert abs(float(gl) - loss) <= (EPS + 2.0 ** -24) * loss + 1e-38
    assert np.all(np.abs(gh - d) <= EPS * scale + (2.0 ** -8 if half else 2.0 ** -23) * np.abs(d) + 1e-38)
    assert not gh[~mask].any()


def test_balance_gradient_against_differences(mx):
    import torch
    rng = np.random.default_rng(1)
    t, e, coef, h = 6, 10, 0.5, 1e-4
    logits = rng.normal(0, 1, (t, e)).astype(np.float32)
    counts = rng.integers(1, 9, e).astype(np.int32)
    _, w = mx.moe_balance_loss(to_dev(logits), to_dev(counts), coef)
    d = mx.moe_balance_loss_grad(to_dev(logits), w, torch.ones(1, device="cuda")).cpu().numpy()
    for i in range(t):
        for j in range(e):
            up, down = logits.astype(np.float64), logits.astype(np.float64)
            up[i, j] += h
            down[i, j] -= h
            slope = (_balance(up, counts, coef, None, 1.0)[0] - _balance(down, counts, coef, None, 1.0)[0]) / (2 * h)
            # central differences: h^2 / 6 times a third derivative of at most 2 max(w) here, and float64 noise
            assert abs(d[i, j] - slope) <= h * h * w.max().item() + 1e-6 * w.max().item()


def test_balance_loss_without_tokens_or_choices(mx):
    import torch
    counts = torch.ones(5, dtype=torch.int32, device="cuda")
    loss, w = mx.moe_balance_loss(torch.empty((0, 5), device="cuda"), counts, 0.1)
    assert float(loss) == 0 and not w.any()
    x = torch.randn((9, 5), device="cuda")
    for c, m in ((counts * 0, None), (counts, torch.zeros(9, dtype=torch.bool, device="cuda"))):
        loss, w = mx.moe_balance_loss(x, c, 0.1, mask=m)
        d = mx.moe_balance_loss_grad(x, w, torch.ones(1, device="cuda"), mask=m)
        assert float(loss) == 0 and not w.any() and not d.any()
    x[3, 2] = float("nan")
    assert torch.isnan(mx.moe_balance_loss(x, counts, 0.1)[0]).item()


def test_refusals(mx):
    import torch
    ids = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    with pytest.raises(mx.MxError):
        mx.moe_route(ids, 1025)
    with pytest.raises(ValueError, match="contiguous"):
        mx.moe_route(ids.t(), 4)
    x, c = torch.zeros((4, 6), device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="per expert"):
        mx.moe_balance_loss(x, c[:5], 0.1)
    with pytest.raises(ValueError, match="per row"):
        mx.moe_balance_loss(x, c, 0.1, mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError, match="bool or uint8"):
        mx.moe_balance_loss(x, c, 0.1, mask=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="grad_loss"):
        mx.moe_balance_loss_grad(x, torch.zeros(6, device="cuda"), torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        mx.moe_balance_loss_grad(x, torch.zeros(6, device="cuda"), torch.ones(1, device="cuda"), dlogits=x[:3])


@pytest.mark.parametrize("t,e,top", [(40, 6, 2), (700, 4, 3)])
def test_router_to_experts(mx, orc, t, e, top):
    """logits -> choices -> packed rows -> quantized tokens -> experts' products -> weighted sum by slots, eagerly and in a
    captured graph that is replayed with other inputs."""
    import torch
    n, k = 200, 384
    qw, sw = zip(*(b128.quant_weight(orc, synth.weight_normal(60 + i, n, k, 0.02)) for i in range(e)))
    qw, sw = np.stack(qw), np.stack(sw)
    qwd, swd = to_dev(qw), to_dev(sw)
    xs = [_bf16(synth.normal(i, t * k).reshape(t, k)) for i in range(3)]
    ls = [np.random.default_rng(i).normal(0, 2, (t, e)).astype(np.float32) for i in range(3)]

    def step(x, logits):
        ids = logits.topk(top, dim=1).indices
        counts, offsets, rows, slots = mx.moe_route(ids, e)
        loss, w = mx.moe_balance_loss(logits, counts, 0.01)
        d = mx.moe_balance_loss_grad(logits, w, torch.ones_like(loss))
        qa, sa = mx.quant_act_b128(x)
        y = mx.gemm_a8w8_b128_grouped(qa, sa, qwd, swd, offsets, rows=rows)
        return ids, slots, y, loss, d
    want = [step(bf16_dev(x), to_dev(l)) for x, l in zip(xs, ls)]
    for (ids, slots, y, _, _), x in zip(want, xs):
        qa, sa = b128.quant_act(orc, x)
        idh, sh, yh = ids.cpu().numpy(), slots.cpu().numpy(), bf16_host(y)
        exact = [b128.gemm(orc, qa, sa, qw[i], sw[i]) for i in range(e)]
        for j in range(top):
            ye = np.stack([exact[idh[r, j]][0][r] for r in range(t)])
            ad = np.stack([exact[idh[r, j]][1][r] for r in range(t)])
            assert b128.accepts(yh[sh[:, j]], ye, ad).all()
    x, logits = bf16_dev(xs[0]), to_dev(ls[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, logits)
    torch.cuda.current_stream().wait_stream(side)
    ids = logits.topk(top, dim=1).indices  # the library's selection stays out of the graph

    def fixed(x, logits):
        counts, offsets, rows, slots = mx.moe_route(ids, e)
        loss, w = mx.moe_balance_loss(logits, counts, 0.01)
        d = mx.moe_balance_loss_grad(logits, w, torch.ones_like(loss))
        qa, sa = mx.quant_act_b128(x)
        return mx.gemm_a8w8_b128_grouped(qa, sa, qwd, swd, offsets, rows=rows), loss, d
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fixed(x, logits)
    for i in (1, 2, 0, 1):
        x.copy_(bf16_dev(xs[i]))
        logits.copy_(to_dev(ls[i]))
        ids.copy_(logits.topk(top, dim=1).indices)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i][2:]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "replay %d" % i
