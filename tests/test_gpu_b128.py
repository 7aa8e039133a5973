"""GPU parity of the block-128 FP8 quantizers, GEMM, grouped GEMM and layer: codes and scales bit for bit, products
against float64 within the rule of b128.py."""
import numpy as np
import pytest

import b128
from block_scaled_precision_act_amd import synth
from parity import bf16_dev, bf16_host, to_dev

pytestmark = pytest.mark.gpu


def _act(seed, m, k):
    """Normal rows with some columns 30 times as large, as BF16 bits."""
    v = synth.normal(seed, m * k).reshape(m, k)
    v[:, ::97] *= 30
    return synth.f64_to_bf16_bits(np.ascontiguousarray(v.reshape(-1))).reshape(m, k)


# ---------------------------------------------------------------- quantizers
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (64, 8192), (1000, 640), (5, 16384)])
def test_quant_act_bit_exact(mx, orc, m, k):
    x = _act(m + k, m, k)
    q, s = mx.quant_act_b128(bf16_dev(x))
    oq, os_ = b128.quant_act(orc, x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), os_.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), oq)


def test_quant_act_special_blocks(mx, orc):
    """Every BF16 pattern as a block's maximum (subnormals, the largest, infinities, NaN), a block of zeros, signed
    zeros and values that lie on code borders."""
    top = np.arange(0x8000, dtype=np.uint32)  # all magnitudes
    x = np.zeros((0x8000, 128), np.uint16)
    x[:, 0] = top
    rng = np.random.default_rng(3)
    frac = rng.integers(0, 0x8000, (0x8000, 100))
    x[:, 10:110] = np.minimum(frac, top[:, None]) | (rng.integers(0, 2, frac.shape) << 15)
    near = np.maximum(top[:, None].astype(np.int64) - rng.integers(0, 0x600, (0x8000, 16)), 0)  # within a few binades
    x[:, 110:126] = near
    x[:, 127] = 0x8000
    q, s = mx.quant_act_b128(bf16_dev(x))
    oq, os_ = b128.quant_act(orc, x)
    nan = np.isnan(os_)
    sg = s.cpu().numpy()
    assert np.array_equal(np.isnan(sg), nan) and nan.sum() == 0x80
    assert np.array_equal(sg[~nan].view(np.uint32), os_[~nan].view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), oq)


@pytest.mark.parametrize("n,k", [(1, 128), (128, 128), (129, 256), (300, 1152), (1000, 2048)])
def test_quant_weight_bit_exact(mx, orc, n, k):
    w = synth.weight_normal(n + k, n, k, 0.02)
    q, s = mx.quant_weight_b128(to_dev(w))
    oq, os_ = b128.quant_weight(orc, w)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), os_.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), oq)


def test_quant_weight_special_blocks(mx, orc):
    w = synth.weight_normal(5, 200, 1280, 1.0)
    w[:128, :128] = 0
    w[0, 128] = np.inf
    w[127, 300] = np.nan
    w[:128, 384:512] *= np.float32(2.0 ** -138)   # subnormal scale, coarsely rounded: quotients pass 448
    w[:128, 512:640] *= np.float32(2.0 ** 120)
    w[:128, 640:768] = 0
    w[3, 640] = np.float32(2.0 ** -149)           # the scale would round to 0: it is 1
    w[:128, 768:896] = np.float32(-0.0)
    q, s = mx.quant_weight_b128(to_dev(w))
    qh, sh = q.cpu().numpy(), s.cpu().numpy()
    assert sh[0, 5] == 1.0 and np.all(qh[:128, 640:768] == 0)
    w[3, 640] = 0  # the oracle's rule has no such case
    oq, os_ = b128.quant_weight(orc, w)
    nan = np.isnan(os_)
    assert np.array_equal(np.isnan(sh), nan) and nan.sum() == 2
    assert np.array_equal(sh[~nan], os_[~nan])
    assert np.array_equal(qh, oq)


# ---------------------------------------------------------------- GEMM
SHAPES = [
    (1, 1, 128), (1, 300, 8192), (2, 7, 256), (5, 1000, 1152), (15, 129, 640), (16, 128, 2048), (17, 64, 384), (31, 200, 4096),
    (33, 100, 128), (48, 577, 1024), (64, 512, 8192), (65, 130, 512), (100, 33, 1280), (128, 256, 2048), (129, 129, 256),
    (200, 1000, 896), (256, 224, 1664), (300, 7, 384), (512, 520, 640), (513, 300, 1152), (777, 1100, 2176), (1025, 513, 256),
    (2049, 260, 128), (1, 7168, 16384), (24, 2100, 16512), (700, 2900, 640),
    (60, 7100, 256), (250, 7100, 640), (500, 7168, 1152), (1000, 7167, 256), (2049, 7168, 1280),  # every tile size
]


def _gemm_case(orc, m, n, k, seed=0):
    qa, sa = b128.quant_act(orc, _act(seed + 7 * m + k, m, k))
    qw, sw = b128.quant_weight(orc, synth.weight_normal(seed + n + k, n, k, 0.02))
    return qa, sa, qw, sw


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_matches_float64(mx, orc, m, n, k):
    import torch
    qa, sa, qw, sw = _gemm_case(orc, m, n, k)
    buf = torch.full((m * n + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = mx.gemm_a8w8_b128(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), y=buf[:m * n].view(m, n))
    ye, ad = b128.gemm(orc, qa, sa, qw, sw)
    b128.check(bf16_host(y), ye, ad)
    assert torch.isnan(buf[m * n:].float()).all(), "wrote behind the output"


@pytest.mark.parametrize("m,n,k", [(3, 200, 512), (70, 200, 512), (600, 300, 384)])
def test_gemm_unaligned_output(mx, orc, m, n, k):
    import torch
    qa, sa, qw, sw = _gemm_case(orc, m, n, k)
    buf = torch.zeros(m * n + 1, dtype=torch.bfloat16, device="cuda")
    y = mx.gemm_a8w8_b128(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), y=buf[1:].view(m, n))
    b128.check(bf16_host(y), *b128.gemm(orc, qa, sa, qw, sw))


@pytest.mark.parametrize("m", [4, 50, 300, 700])
def test_gemm_every_code_and_scale_range(mx, orc, m):
    """All finite codes with scales over 2^-40 .. 2^40; one row and one weight block with a NaN scale, one NaN code: NaN
    exactly where they reach."""
    n, k = 200, 512
    rng = np.random.default_rng(m)
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    qa, qw = codes[rng.integers(0, len(codes), (m, k))], codes[rng.integers(0, len(codes), (n, k))]
    sa = (2.0 ** rng.uniform(-40, 40, (m, k // 128))).astype(np.float32)
    sw = (2.0 ** rng.uniform(-40, 40, ((n + 127) // 128, k // 128))).astype(np.float32)
    sa[m - 1, 1] = np.nan
    sw[1, 2] = np.nan
    qw[5, 17] = 0x7f
    ye, ad = b128.gemm(orc, qa, sa, qw, sw)
    assert np.isnan(ye[:, 5]).all() and np.isnan(ye[m - 1]).all() and np.isnan(ye[:, 128:]).all() and np.isfinite(ye[0, 0])
    y = mx.gemm_a8w8_b128(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw))
    assert b128.accepts(bf16_host(y), ye, ad).all()


@pytest.mark.parametrize("m,n,k", [(1, 384, 1024), (1, 1, 128), (2, 37, 384), (2, 300, 5120), (1, 50, 16384), (2, 100, 16384),
                                   (1, 130, 65536), (3, 384, 1024), (40, 384, 1024), (129, 384, 1024), (640, 384, 1024)])
def test_layer_is_quantizer_and_gemm(mx, orc, m, n, k):
    import torch
    x = _act(m, m, k)
    qw, sw = b128.quant_weight(orc, synth.weight_normal(m, n, k, 0.02))
    xd, qwd, swd = bf16_dev(x), to_dev(qw), to_dev(sw)
    y = mx.linear_a8w8_b128(xd, qwd, swd)
    qa, sa = b128.quant_act(orc, x)
    b128.check(bf16_host(y), *b128.gemm(orc, qa, sa, qw, sw))
    again = mx.linear_a8w8_b128(xd, qwd, swd)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))


def test_empty_shapes(mx):
    import torch
    q, s = mx.quant_act_b128(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    qw, sw = mx.quant_weight_b128(torch.ones((5, 256), device="cuda"))
    assert mx.gemm_a8w8_b128(q, s, qw, sw).shape == (0, 5)
    y = mx.gemm_a8w8_b128_grouped(q, s, qw.view(1, 5, 256), sw.view(1, 1, 2), torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 5)


def test_refuses_wrong_shapes_and_types(mx):
    import torch
    qa, sa = torch.zeros((4, 256), dtype=torch.uint8, device="cuda"), torch.ones((4, 2), device="cuda")
    qw, sw = torch.zeros((130, 256), dtype=torch.uint8, device="cuda"), torch.ones((2, 2), device="cuda")
    for bad in ((qa, sa[:3].contiguous(), qw, sw), (qa, sa, qw, sw[:1].contiguous()), (qa, sa, qw[:, :128].contiguous(), sw)):
        with pytest.raises(ValueError):
            mx.gemm_a8w8_b128(*bad)
    with pytest.raises(ValueError, match="contiguous"):
        mx.gemm_a8w8_b128(qa, sa, qw[::2], sw[:1])
    with pytest.raises(ValueError, match="shape"):
        mx.gemm_a8w8_b128(qa, sa, qw, sw, y=torch.empty((4, 131), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mx.MxError):
        mx.quant_act_b128(torch.zeros((2, 192), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mx.gemm_a8w8_b128_grouped(qa, sa, qw.view(1, 130, 256), sw.view(1, 2, 2), torch.zeros(3, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- grouped
def _experts(orc, g, n, k):
    qw, sw = zip(*(b128.quant_weight(orc, synth.weight_normal(50 + i, n, k, 0.02)) for i in range(g)))
    return np.stack(qw), np.stack(sw)


def _check_groups(orc, y, sizes, qa, sa, qw, sw, rows):
    yh, at = bf16_host(y), 0
    for e, c in enumerate(sizes):
        r = rows[at:at + c]
        ok_row = (r >= 0) & (r < qa.shape[0])
        ye, ad = b128.gemm(orc, qa[np.where(ok_row, r, 0)], sa[np.where(ok_row, r, 0)], qw[e], sw[e])
        ye[~ok_row], ad[~ok_row] = 0, 0
        ok = b128.accepts(yh[at:at + c], ye, ad)
        assert ok.all(), "group %d: %d outside tolerance" % (e, (~ok).sum())
        at += c


@pytest.mark.parametrize("sizes,n,k", [
    ([0, 1, 17, 0, 5], 300, 512), ([3], 129, 256), ([1] * 20, 64, 384), ([40, 0, 33, 64, 2], 200, 1152),
    ([200, 3, 0, 129], 130, 640), ([0, 0, 500], 257, 256), ([700, 1000, 0, 33], 300, 384), ([0, 0], 16, 128),
    ([1300, 2, 600], 260, 256),
    ([10, 0, 5, 3] * 2, 3000, 640), ([10, 0, 20, 31], 6000, 640), ([40, 0, 33, 64, 2], 4100, 384), ([200, 3, 0, 129], 4100, 1152), ([700, 1000, 0, 33], 4100, 256),
])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_matches_float64(mx, orc, sizes, n, k, gather):
    import torch
    total, extra = sum(sizes), 3  # rows behind the last group stay as they were
    qw, sw = _experts(orc, len(sizes), n, k)
    rng = np.random.default_rng(total + n)
    arows = 50 if gather else total + extra
    qa, sa = b128.quant_act(orc, _act(total + k, arows, k))
    rows = rng.integers(0, arows, total + extra).astype(np.int32) if gather else np.arange(total + extra, dtype=np.int32)
    if gather and total > 4:
        rows[[1, total - 1]] = [-1, arows]  # no such row: zeros
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = torch.full((total + extra, n), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.gemm_a8w8_b128_grouped(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), to_dev(off), rows=to_dev(rows) if gather else None,
                              y=y)
    _check_groups(orc, y, sizes, qa, sa, qw, sw, rows)
    assert (y[total:].float() == 7.0).all()


# tiles of all four heights (one, two and three of them to a group); more groups than a wave's lanes, few and many rows each
@pytest.mark.parametrize("sizes,n,k", [
    ([60, 120, 190, 250, 300, 0, 600, 30], 10000, 384), ([64, 65, 128, 129, 192, 193, 256, 257], 10000, 128),
    ([(37 * i) % 260 for i in range(70)], 2048, 128), ([1] * 70 + [0] * 30 + [3] * 40, 64, 384), ([20, 5] * 40, 2000, 128),
])
def test_grouped_heights_and_many_groups(mx, orc, sizes, n, k):
    import torch
    total, arows = sum(sizes), 40
    qw, sw = _experts(orc, len(sizes), n, k)
    qa, sa = b128.quant_act(orc, _act(total + k, arows, k))
    rows = np.random.default_rng(total).integers(0, arows, total).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = torch.full((total, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    mx.gemm_a8w8_b128_grouped(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), to_dev(off), rows=to_dev(rows), y=y)
    _check_groups(orc, y, sizes, qa, sa, qw, sw, rows)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 40], [-3, 4, 9, 1000], [0, 0, 0, 0], [2, 6, 6, 20]])
@pytest.mark.parametrize("t", [20, 400])
def test_grouped_offsets_out_of_order_or_range(mx, orc, offsets, t):
    """Each group is what its clamped offsets say; rows of no group stay as they were."""
    import torch
    n, k, g = 130, 256, 3
    qw, sw = _experts(orc, g, n, k)
    qa, sa = b128.quant_act(orc, _act(t, t, k))
    y = torch.full((t, n), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.gemm_a8w8_b128_grouped(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), to_dev(np.array(offsets, np.int32)), y=y)
    yh = bf16_host(y)
    c = np.clip(offsets, 0, t)
    owners = [[e for e in range(g) if c[e] <= r < c[e + 1]] for r in range(t)]
    for r in range(t):
        if not owners[r]:
            assert (yh[r] == 7.0).all()
        elif len(owners[r]) == 1:
            e = owners[r][0]
            assert b128.accepts(yh[r:r + 1], *b128.gemm(orc, qa[r:r + 1], sa[r:r + 1], qw[e], sw[e])).all()


def test_other_stream_and_graph_replays(mx, orc):
    """The layer and the grouped product on a side stream, and captured: every replay equals the eager result on the
    inputs of that replay, with eager work between."""
    import torch
    m, n, k, g = 40, 300, 640, 4
    qw, sw = _experts(orc, g, n, k)
    qw, sw = to_dev(qw), to_dev(sw)
    off = to_dev(np.array([0, 10, 10, 37, m], np.int32))
    xs = [bf16_dev(_act(100 + i, m, k)) for i in range(4)]

    def both(x):
        qa, sa = mx.quant_act_b128(x)
        return mx.linear_a8w8_b128(x, qw[1], sw[1]), mx.gemm_a8w8_b128_grouped(qa, sa, qw, sw, off)
    want = [both(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(xs[0])
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want[0]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        both(xs[(i + 1) % 4])
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "replay %d" % i


def test_calls_on_two_streams_at_once(mx, orc):
    """Layers and grouped products in flight on two streams, each with its own inputs, do not disturb each other."""
    import torch
    n, k, g = 700, 2176, 3
    qw, sw = _experts(orc, g, n, k)
    qw, sw = to_dev(qw), to_dev(sw)
    work = [(bf16_dev(_act(200 + m, m, k)), to_dev(np.array([0, m // 3, m // 2, m], np.int32))) for m in (2, 50, 333, 900)]

    def run(x, off):
        qa, sa = mx.quant_act_b128(x)
        return mx.linear_a8w8_b128(x, qw[0], sw[0]), mx.gemm_a8w8_b128_grouped(qa, sa, qw, sw, off)
    want = [run(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(run(*work[(i * 3 + i // 4) % 4]))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        for a, b in zip(pair, want[(i * 3 + i // 4) % 4]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "call %d" % i


@pytest.mark.parametrize("m", [2, 60, 300])
def test_infinite_scales_stay_infinite(mx, m):
    """An infinite scale gives infinities where its block's sum is not 0, also where K ends inside a step of the kernels."""
    import torch
    n, k = 130, 640
    q = torch.full((m, k), 0x38, dtype=torch.uint8, device="cuda")   # 1.0
    qw = torch.full((n, k), 0x38, dtype=torch.uint8, device="cuda")
    sa, sw = torch.ones((m, k // 128), device="cuda"), torch.ones((2, k // 128), device="cuda")
    sa[0, 4] = float("inf")
    sw[1, 4] = float("inf")
    y = mx.gemm_a8w8_b128(q, sa, qw, sw).float()
    assert torch.isinf(y[0]).all() and torch.isinf(y[:, 128:]).all() and (y[1:, :128] == 640).all()
