"""int8 linear layer and mixture-of-experts layer without a GPU: the weight
quantiser, the packer, size rules and every refusal of the C ABI and the
binding (all of them before a HIP call)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import weight_only_fp6_amd as fp6
from weight_only_fp6_amd import synth

from _operators_ref import int8_codes

L = fp6.lib
A = 1 << 20          # an aligned address; never dereferenced, every check fails first
OK, NULL, SHAPE, ALIGN, SIZE, VALUE = 0, 1, 2, 3, 6, 8


# --- weight quantiser -------------------------------------------------------
@pytest.mark.parametrize("shape", [(1, 1), (3, 15), (5, 16), (4, 17), (7, 300)])
def test_int8_rows_against_64_bits(shape):
    W = synth.weights(*shape, seed=11 + shape[1])
    q, s = fp6.int8_quantize_rows(W)
    qr, sr = int8_codes(W)
    assert q.shape == (shape[0], fp6.int8_padded_k(shape[1]))
    assert np.array_equal(q[:, : shape[1]], qr) and not q[:, shape[1]:].any()
    assert np.array_equal(s.astype(np.float64), sr)


def test_int8_rows_ties_zero_rows_and_range():
    W = np.zeros((4, 256), np.float32)
    W[1, :2] = [2.0, 1.0]                       # 127 * 1/2 = 63.5: a tie, to the even 64
    W[2, :255] = np.arange(-127, 128) * 3.0     # every code, exactly
    W[3, :2] = [3e38, -3e38]
    q, s = fp6.int8_quantize_rows(W)
    assert s[0] == 0 and not q[0].any()
    assert list(q[1, :2]) == [127, 64]
    assert np.array_equal(q[2, :255], np.arange(-127, 128))
    assert list(q[3, :2]) == [127, -127]
    rng = np.random.default_rng(3)
    W = rng.standard_normal((8, 64)).astype(np.float32)
    q, _ = fp6.int8_quantize_rows(W)
    for n in range(8):                          # the rational definition
        a = Fraction(float(np.abs(W[n]).max()))
        assert [int(round(127 * Fraction(float(w)) / a)) for w in W[n]] == list(q[n])


def test_int8_rows_refusals():
    W = np.ones((2, 3), np.float32)
    for bad in (np.inf, -np.inf, np.nan):
        V = W.copy()
        V[1, 2] = bad
        with pytest.raises(fp6.FP6Error, match="FP6_E_VALUE"):
            fp6.int8_quantize_rows(V)
    with pytest.raises(ValueError):
        fp6.int8_quantize_rows(W[0])
    assert L.fp6_int8_quantize_rows(None, 1, 1, A, A) == NULL
    assert L.fp6_int8_quantize_rows(A, 0, 16, A, A) == SHAPE
    assert L.fp6_int8_quantize_rows(A, 1, 131057, A, A) == SHAPE


def test_int8_sizes():
    assert [fp6.int8_padded_k(k) for k in (1, 16, 17, 131056)] == [16, 16, 32, 131056]
    assert [fp6.int8_padded_k(k) for k in (0, -5, 131057)] == [0, 0, 0]
    assert L.fp6_int8_workspace_bytes(3, 17) == 3 * 32 + 12
    assert L.fp6_int8_workspace_bytes(0, 17) == 0 and L.fp6_int8_workspace_bytes(1, 0) == 0


# --- C ABI refusals ---------------------------------------------------------
def test_int8_quantize_tokens_refusals():
    f = L.fp6_int8_quantize_tokens
    assert f(0, None, 8, 0, 8, None, None, None) == OK
    assert f(2, A, 8, 1, 8, A, A, None) == VALUE
    assert f(0, A, 7, 1, 8, A, A, None) == SHAPE
    assert f(0, A, 8, -1, 8, A, A, None) == SHAPE
    assert f(0, A, 8, 1, 0, A, A, None) == SHAPE
    assert f(0, A, 1 << 20, 1 << 24, 1 << 16, A, A, None) == SHAPE
    for i in (1, 5, 6):
        args = [0, A, 8, 1, 8, A, A, None]
        args[i] = None
        assert f(*args) == NULL
    assert f(0, A + 1, 8, 1, 8, A, A, None) == ALIGN
    assert f(0, A, 8, 1, 8, A + 8, A, None) == ALIGN
    assert f(0, A, 8, 1, 8, A, A + 2, None) == ALIGN


def test_int8_linear_refusals():
    f = L.fp6_int8_linear
    good = [A, A, A, A, None, 0, A, 4, 5, 32, None]
    assert f(*good[:7], 0, 5, 32, None) == OK
    for i, v, st in [(5, 2, VALUE), (5, -1, VALUE), (7, -1, SHAPE), (8, 0, SHAPE), (9, 0, SHAPE), (9, 24, SHAPE),
                     (9, 131072, SHAPE), (7, 1 << 25, SHAPE), (0, None, NULL), (1, None, NULL), (2, None, NULL),
                     (3, None, NULL), (6, None, NULL), (0, A + 8, ALIGN), (2, A + 4, ALIGN), (6, A + 2, ALIGN),
                     (1, A + 2, ALIGN), (3, A + 1, ALIGN), (4, A + 1, ALIGN)]:
        args = list(good)
        args[i] = v
        assert f(*args) == st, (i, v)
    assert f(A, A, A, A, None, 0, A, 1 << 24, 1 << 24, 16, None) == SHAPE   # M*N


def test_int8_linear_tokens_refusals():
    f = L.fp6_int8_linear_tokens
    need = L.fp6_int8_workspace_bytes(4, 20)
    good = [0, A, 20, A, A, None, 1, A, 4, 5, 20, A, need, None]
    for i, v, st in [(0, 3, VALUE), (6, 3, VALUE), (2, 19, SHAPE), (10, 0, SHAPE), (9, 0, SHAPE), (1, None, NULL),
                     (3, None, NULL), (4, None, NULL), (7, None, NULL), (11, None, NULL), (1, A + 1, ALIGN),
                     (3, A + 8, ALIGN), (7, A + 8, ALIGN), (11, A + 8, ALIGN), (4, A + 2, ALIGN), (5, A + 1, ALIGN),
                     (12, need - 1, SIZE)]:
        args = list(good)
        args[i] = v
        assert f(*args) == st, (i, v)
    args = list(good)
    args[8] = 0
    assert f(*args) == OK


def test_moe_sizes_and_refusals():
    W = L.fpx_moe_workspace_bytes
    assert W(1, 8, 2, 1024, 512) > 0
    assert W(1, 2, 8, 1024, 512) > 0     # a shard with fewer experts than choices
    for bad in [(0, 8, 2, 1024, 512), (1, 0, 1, 1024, 512), (1, 513, 2, 1024, 512), (1, 8, 0, 1024, 512),
                (1, 64, 17, 1024, 512), (1, 8, 2, 1000, 512), (1, 8, 2, 1024, 128),
                (1, 8, 2, 0, 512), (65537, 8, 2, 1024, 512), (1, 8, 2, 1 << 20, 1 << 20)]:
        assert W(*bad) == 0, bad
    need = W(4, 8, 2, 1024, 512)
    ex = [0, A, A, A, A, A, A, A, A, 4, 8, 2, 1024, 512, A, need, None]
    for i, v, st in [(0, 4, VALUE), (0, -1, VALUE), (9, -1, SHAPE), (11, 17, SHAPE), (12, 100, SHAPE),
                     (13, 300, SHAPE), (14, None, NULL), (14, A + 16, ALIGN), (15, need - 1, SIZE)] + \
            [(i, None, NULL) for i in range(1, 9)] + \
            [(1, A + 8, ALIGN), (2, A + 2, ALIGN), (3, A + 2, ALIGN), (4, A + 8, ALIGN), (5, A + 1, ALIGN),
             (6, A + 8, ALIGN), (7, A + 1, ALIGN), (8, A + 8, ALIGN)]:
        args = list(ex)
        args[i] = v
        assert L.fpx_moe_experts(*args) == st, (i, v)
    args = list(ex)
    args[9] = 0
    assert L.fpx_moe_experts(*args) == OK
    ly = [0, A, A, A, A, A, A, 1, A, A, A, 4, 8, 2, 1024, 512, A, need, None]
    for i, v, st in [(7, 2, VALUE), (2, None, NULL), (2, A + 8, ALIGN), (9, None, NULL), (17, need - 1, SIZE),
                     (13, 9, SHAPE)]:
        args = list(ly)
        args[i] = v
        assert L.fpx_moe_layer(*args) == st, (i, v)
    args = list(ly)
    args[11] = 0
    assert L.fpx_moe_layer(*args) == OK


# --- binding ----------------------------------------------------------------
def test_moe_prepack_is_prepack_of_each_expert():
    rng = np.random.default_rng(1)
    for fmt in fp6.FORMATS:
        codes = rng.integers(0, 1 << fp6.bits(fmt), (3, 32, 256), dtype=np.uint8)
        scales = rng.uniform(0.01, 1, (3, 32)).astype(np.float16)
        got = fp6.moe_prepack(codes, scales, fmt)
        for e in range(3):
            assert np.array_equal(got[e], fp6.prepack(codes[e], scales[e], fmt))
    with pytest.raises(fp6.FP6Error, match="FP6_E_CODE"):
        fp6.moe_prepack(np.full((2, 16, 256), 255, np.uint8), np.ones((2, 16), np.float16))
    with pytest.raises(ValueError):
        fp6.moe_prepack(codes[0], scales[0])
    with pytest.raises(ValueError):
        fp6.moe_prepack(codes, scales, "e5m2")


def test_int8_binding_refuses_on_the_cpu():
    X = torch.zeros(4, 20, dtype=torch.float16)
    W = torch.zeros(6, 32, dtype=torch.int8)
    sw = torch.ones(6)
    with pytest.raises(ValueError, match="GPU"):
        fp6.int8_quantize_tokens(X)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        fp6.int8_quantize_tokens(X.float())
    with pytest.raises(ValueError, match="side by side"):
        fp6.int8_quantize_tokens(torch.zeros(20, 4, dtype=torch.float16).t())
    with pytest.raises(ValueError, match="overlap"):
        fp6.int8_quantize_tokens(X[:1].expand(4, 20))
    Q = torch.zeros(4, 32, dtype=torch.int8)
    with pytest.raises(ValueError, match="x_scales"):
        fp6.int8_linear(Q, W, sw)
    with pytest.raises(ValueError, match="x_scales"):
        fp6.int8_linear(X, W, sw, x_scales=torch.ones(4))
    with pytest.raises(ValueError, match="X must be"):
        fp6.int8_linear(Q[:, :16].contiguous(), W, sw, x_scales=torch.ones(4))
    with pytest.raises(ValueError, match="GPU"):
        fp6.int8_linear(Q, W, sw, x_scales=torch.ones(4))
    with pytest.raises(ValueError, match="W must be"):
        fp6.int8_linear(Q, W[0], sw, x_scales=torch.ones(4))


def test_moe_binding_refuses_on_the_cpu():
    X = torch.zeros(2, 256, dtype=torch.float16)
    s13, s2 = torch.ones(4, 512, dtype=torch.float16), torch.ones(4, 256, dtype=torch.float16)
    w13 = torch.zeros(4, fp6.packed_bytes(512, 256), dtype=torch.uint8)
    w2 = torch.zeros(4, fp6.packed_bytes(256, 256), dtype=torch.uint8)
    ids, w = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    with pytest.raises(ValueError, match="GPU"):
        fp6.moe_experts(X, ids, w, w13, s13, w2, s2)
    with pytest.raises(ValueError, match="X must be"):
        fp6.moe_experts(X[0], ids, w, w13, s13, w2, s2)
    with pytest.raises(ValueError, match="unknown weight format"):
        fp6.moe_experts(X, ids, w, w13, s13, w2, s2, fmt="e4m3")
    with pytest.raises(ValueError, match="gate_up_scales"):
        fp6.moe_layer(X, X, w13, s13[0], w2, s2, 1)
