"""Block-128 FP8 and expert-routing entry points: argument errors are reported on the host before anything
reaches a device.  Runs without a GPU (no kernel is launched here)."""
import os

import pytest

FAKE = 0x10000  # a non-null, 64K-aligned address that is never dereferenced


@pytest.fixture(scope="module")
def mx():
    from block_scaled_precision_act_amd import build, mxgemm
    if not os.path.exists(mxgemm.LIB_PATH):
        build.build(verbose=False)
    return mxgemm


def test_quantizers(mx):
    for f in (mx.b128_quant_act_fp8, mx.b128_quant_weight_f32):
        assert f(FAKE, -1, 128, FAKE, FAKE) == mx.MX_ERROR_INVALID_VALUE
        assert f(FAKE, 4, 64, FAKE, FAKE) == mx.MX_ERROR_UNSUPPORTED_SHAPE
        assert f(FAKE, 4, 192, FAKE, FAKE) == mx.MX_ERROR_UNSUPPORTED_SHAPE
        assert f(FAKE, 4, 0, FAKE, FAKE) == mx.MX_ERROR_UNSUPPORTED_SHAPE
        assert f(FAKE, 1 << 40, 128, FAKE, FAKE) == mx.MX_ERROR_UNSUPPORTED_SHAPE
        assert f(None, 4, 128, FAKE, FAKE) == mx.MX_ERROR_INVALID_VALUE
        assert f(FAKE, 4, 128, None, FAKE) == mx.MX_ERROR_INVALID_VALUE
        assert f(FAKE, 4, 128, FAKE, None) == mx.MX_ERROR_INVALID_VALUE
        assert f(FAKE + 8, 4, 128, FAKE, FAKE) == mx.MX_ERROR_MISALIGNED
        assert f(FAKE, 4, 128, FAKE + 2, FAKE) == mx.MX_ERROR_MISALIGNED
        assert f(FAKE, 4, 128, FAKE, FAKE + 2) == mx.MX_ERROR_MISALIGNED
        assert f(None, 0, 128, None, None) == mx.MX_SUCCESS


def test_gemm(mx):
    f = mx.gemm_a8w8_b128_bf16
    five = (FAKE,) * 5
    assert f(*five, -1, 4, 128) == mx.MX_ERROR_INVALID_VALUE
    assert f(*five, 4, -1, 128) == mx.MX_ERROR_INVALID_VALUE
    assert f(*five, 4, 4, 64) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    assert f(*five, 1 << 32, 4, 128) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    assert f(*five, 4, 4, 1 << 23) == mx.MX_ERROR_UNSUPPORTED_SHAPE           # a tile's rows past 32-bit offsets
    assert f(*five, 1 << 30, 1 << 30, 128) == mx.MX_ERROR_UNSUPPORTED_SHAPE   # more tiles than a grid holds
    for i in range(5):
        assert f(*(None if j == i else FAKE for j in range(5)), 4, 4, 128) == mx.MX_ERROR_INVALID_VALUE
    for i, off in enumerate((8, 2, 8, 2, 1)):
        assert f(*(FAKE + (off if j == i else 0) for j in range(5)), 4, 4, 128) == mx.MX_ERROR_MISALIGNED
    assert f(*(None,) * 5, 0, 4, 128) == mx.MX_SUCCESS
    assert f(*(None,) * 5, 4, 0, 128) == mx.MX_SUCCESS


def test_layer(mx):
    f = mx.linear_a8w8_b128_bf16
    need = mx.linear_a8w8_b128_workspace_bytes(40, 64, 256)
    assert need > 0 and mx.linear_a8w8_b128_workspace_bytes(0, 64, 256) == 0 and mx.linear_a8w8_b128_workspace_bytes(4, 4, 100) == 0
    four = (FAKE,) * 4
    assert f(*four, -1, 64, 256) == mx.MX_ERROR_INVALID_VALUE
    assert f(*four, 40, 64, 200) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    assert f(*four, 40, 64, 1 << 23, FAKE, 1 << 40) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    for i in range(4):
        assert f(*(None if j == i else FAKE for j in range(4)), 40, 64, 256, FAKE, need) == mx.MX_ERROR_INVALID_VALUE
    for i, off in enumerate((8, 8, 2, 1)):
        assert f(*(FAKE + (off if j == i else 0) for j in range(4)), 40, 64, 256, FAKE, need) == mx.MX_ERROR_MISALIGNED
    assert f(*four, 40, 64, 256) == mx.MX_ERROR_WORKSPACE
    assert f(*four, 40, 64, 256, FAKE, need - 1) == mx.MX_ERROR_WORKSPACE
    assert f(*four, 40, 64, 256, FAKE + 8, need) == mx.MX_ERROR_MISALIGNED
    assert f(*(None,) * 4, 0, 64, 256) == mx.MX_SUCCESS


def test_grouped_gemm(mx):
    f = mx.gemm_a8w8_b128_grouped_bf16
    assert f(FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None, -1, 4, 16, 128) == mx.MX_ERROR_INVALID_VALUE
    assert f(FAKE, FAKE, -1, FAKE, FAKE, FAKE, FAKE, None, 2, 4, 16, 128) == mx.MX_ERROR_INVALID_VALUE
    assert f(FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None, 65536, 4, 16, 128) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    assert f(FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None, 2, 4, 16, 96) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    assert f(FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE, None, 2, 4, 16, 128) == mx.MX_ERROR_INVALID_VALUE  # fewer rows than Y
    assert f(FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 16, 128) == mx.MX_ERROR_INVALID_VALUE  # no row to gather
    assert f(FAKE, FAKE, 1 << 25, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 16, 128) == mx.MX_ERROR_UNSUPPORTED_SHAPE  # 32-bit offsets
    for i in range(6):
        p = [None if j == i else FAKE for j in range(6)]
        assert f(p[0], p[1], 4, p[2], p[3], p[4], p[5], None, 2, 4, 16, 128) == mx.MX_ERROR_INVALID_VALUE
    for i, off in enumerate((8, 2, 8, 2, 1, 2, 2)):
        p = [FAKE + (off if j == i else 0) for j in range(7)]
        assert f(p[0], p[1], 4, p[2], p[3], p[4], p[5], p[6], 2, 4, 16, 128) == mx.MX_ERROR_MISALIGNED
    for G, T, N in ((0, 4, 16), (2, 0, 16), (2, 4, 0)):
        assert f(*(None,) * 2, 0, *(None,) * 5, G, T, N, 128) == mx.MX_SUCCESS


def test_route(mx):
    def f(ids=FAKE, size=8, T=4, top=2, E=8, counts=FAKE, offsets=FAKE, rows=FAKE, slots=FAKE, ws=None, wsb=0):
        return mx.lib().moe_route(ids, size, T, top, E, counts, offsets, rows, slots, ws, wsb, None)
    for bad in (dict(T=-1), dict(top=-1), dict(size=2), dict(ids=None), dict(counts=None), dict(offsets=None), dict(rows=None),
                dict(slots=None)):
        assert f(**bad) == mx.MX_ERROR_INVALID_VALUE, bad
    for bad in (dict(E=0), dict(E=1025), dict(T=1 << 24, top=2)):
        assert f(**bad) == mx.MX_ERROR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(ids=FAKE + 4), dict(ids=FAKE + 2, size=4), dict(counts=FAKE + 2), dict(offsets=FAKE + 2),
                dict(rows=FAKE + 2), dict(slots=FAKE + 2)):
        assert f(**bad) == mx.MX_ERROR_MISALIGNED, bad
    big = dict(T=1 << 16, top=8, E=256)
    need = mx.moe_route_workspace_bytes(1 << 16, 8, 256)
    assert need > 0 and mx.moe_route_workspace_bytes(1024, 8, 8) == 0 and mx.moe_route_workspace_bytes(-1, 2, 8) == 0
    assert f(**big) == mx.MX_ERROR_WORKSPACE
    assert f(**big, ws=FAKE, wsb=need - 1) == mx.MX_ERROR_WORKSPACE
    assert f(**big, ws=FAKE + 4, wsb=need) == mx.MX_ERROR_MISALIGNED


def test_balance_loss(mx):
    def f(logits=FAKE, dtype=0, T=4, E=8, counts=FAKE, loss=FAKE, w=FAKE, ws=None, wsb=0):
        return mx.lib().moe_balance_loss(logits, dtype, T, E, counts, None, 0.1, loss, w, ws, wsb, None)
    for bad in (dict(T=-1), dict(dtype=2), dict(logits=None), dict(counts=None), dict(loss=None), dict(w=None)):
        assert f(**bad) == mx.MX_ERROR_INVALID_VALUE, bad
    for bad in (dict(E=0), dict(E=1025), dict(T=1 << 31)):
        assert f(**bad) == mx.MX_ERROR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(logits=FAKE + 2), dict(logits=FAKE + 1, dtype=1), dict(counts=FAKE + 2), dict(loss=FAKE + 2), dict(w=FAKE + 2)):
        assert f(**bad) == mx.MX_ERROR_MISALIGNED, bad
    need = mx.moe_balance_loss_workspace_bytes(100000, 64)
    assert need > 0 and mx.moe_balance_loss_workspace_bytes(1, 8) == 0
    assert f(T=100000, E=64) == mx.MX_ERROR_WORKSPACE
    assert f(T=100000, E=64, ws=FAKE, wsb=need - 1) == mx.MX_ERROR_WORKSPACE

    def g(logits=FAKE, dtype=0, T=4, E=8, w=FAKE, grad=FAKE, d=FAKE):
        return mx.lib().moe_balance_loss_grad(logits, dtype, T, E, w, None, grad, d, None)
    for bad in (dict(T=-1), dict(dtype=-1), dict(logits=None), dict(w=None), dict(grad=None), dict(d=None)):
        assert g(**bad) == mx.MX_ERROR_INVALID_VALUE, bad
    assert g(E=1025) == mx.MX_ERROR_UNSUPPORTED_SHAPE
    for bad in (dict(logits=FAKE + 2), dict(w=FAKE + 2), dict(grad=FAKE + 2), dict(d=FAKE + 2), dict(d=FAKE + 1, dtype=1)):
        assert g(**bad) == mx.MX_ERROR_MISALIGNED, bad
    assert g(T=0, logits=None, w=None, grad=None, d=None) == mx.MX_SUCCESS


def test_tensor_helpers_refuse_host_tensors_and_wrong_types(mx):
    import torch
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        mx.quant_act_b128(x)
    with pytest.raises(TypeError, match="bfloat16"):
        mx.quant_act_b128(x.float())
    with pytest.raises(TypeError, match="float32"):
        mx.quant_weight_b128(x)
    with pytest.raises(TypeError, match="int32 or int64"):
        mx.moe_route(x, 4)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mx.moe_balance_loss(x.half(), x, 0.1)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mx.moe_balance_loss_grad(x.double(), x, x)
    u = torch.zeros((2, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        mx.gemm_a8w8_b128(u, x.float(), u, x.float())
