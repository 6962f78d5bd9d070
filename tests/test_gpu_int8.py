"""int8 quantiser and linear layer against 64-bit references (needs an MI355X)."""

import numpy as np
import pytest

from _operators_ref import int8_codes, int8_product

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import weight_only_fp6_amd as fp6  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _tokens(M, K, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K + pad), generator=g)
    x[:, :: max(1, K // 5)] *= 20
    return x.to(DT[dtype]).to(DEV)[:, :K]


def _codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def _f64(t):
    return t.detach().cpu().double().numpy()


# --- quantiser --------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (3, 7, 0), (2, 16, 8), (5, 17, 3), (4, 255, 1), (1, 1024, 0),
                                     (7, 1025, 0), (33, 2048, 8), (3, 8192, 16), (2, 9001, 0), (1, 131056, 0),
                                     (9, 512, 1), (6, 513, 0), (5, 2049, 3), (2, 4096, 5), (3, 4097, 0), (2, 16384, 0),
                                     (2, 16385, 7)])
def test_quantize_tokens(dtype, M, K, pad):
    X = _tokens(M, K, dtype, 100 * M + K, pad)
    q, s = fp6.int8_quantize_tokens(X)
    qr, sr = int8_codes(_f64(X))
    kp = fp6.int8_padded_k(K)
    assert q.shape == (M, kp) and q.dtype == torch.int8
    assert np.array_equal(_f64(q)[:, :K], qr)
    assert not q[:, K:].any()
    assert np.array_equal(_f64(s), sr)


@pytest.mark.parametrize("top", [1.0, 65504.0, 127.0, 254.0, 2047.0, 1.7e-3, 6e-8, 3.3e-5])
def test_quantize_every_fp16_value(top):
    # Every fp16 number up to `top`: all ties and near-ties of that divisor.
    bits = np.arange(0, 0x7C00, dtype=np.uint16).view(np.float16)
    top = np.float16(top)
    v = bits[bits <= top]
    v = np.concatenate([v, -v])
    X = torch.from_numpy(v[None, :].copy()).to(DEV)
    q, _ = fp6.int8_quantize_tokens(X)
    assert np.array_equal(_f64(q)[:, : v.size], int8_codes(v[None, :])[0])


@pytest.mark.parametrize("top", [1.0, 3.38e38, 254.0, 1.5e-39, 1e-38, 9.2e-41])
def test_quantize_every_bf16_value(top):
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = bits[bits.float() <= top]
    X = torch.cat([v, -v])[None, :].to(DEV)
    q, s = fp6.int8_quantize_tokens(X)
    qr, sr = int8_codes(_f64(X))
    assert np.array_equal(_f64(q)[:, : X.shape[1]], qr)
    assert np.array_equal(_f64(s), sr)


def test_quantize_zero_and_non_finite_rows():
    X = torch.randn(6, 40, dtype=torch.float16, device=DEV)
    X[1] = 0
    X[2, 5] = float("inf")
    X[3, 39] = float("nan")
    X[4, 0] = float("-inf")
    for x in (X, X.bfloat16()):
        q, s = fp6.int8_quantize_tokens(x)
        assert s[1] == 0 and torch.isnan(s[2:5]).all() and torch.isfinite(s[[0, 5]]).all()
        assert not q[1:5].any()
        W = torch.ones(3, 48, dtype=torch.int8, device=DEV)
        y = fp6.int8_linear(q, W, torch.ones(3, device=DEV), x_scales=s)
        assert (y[1] == 0).all() and torch.isnan(y[2:5]).all() and torch.isfinite(y[[0, 5]]).all()


def test_quantize_leaves_what_is_behind_its_outputs():
    buf = torch.full((6, 48), 77, dtype=torch.int8, device=DEV)
    sb = torch.full((6,), 5.0, device=DEV)
    fp6.int8_quantize_tokens(_tokens(4, 33, "fp16", 1), out=buf[:4], scales=sb[:4])
    assert (buf[4:] == 77).all() and (sb[4:] == 5).all() and not buf[:4, 33:].any()


# --- linear -----------------------------------------------------------------
SHAPES = [(1, 1, 16), (1, 16, 64), (1, 250, 1024), (2, 17, 48), (4, 4096, 2064), (15, 63, 272), (16, 33, 4096),
          (16, 5000, 512), (17, 20, 80), (31, 129, 1040), (32, 64, 2048), (33, 16, 16), (64, 200, 640), (65, 31, 336),
          (100, 3, 96), (128, 260, 1152), (200, 511, 784), (257, 300, 4112), (300, 1030, 256), (513, 258, 128),
          (1000, 770, 1312), (2000, 2100, 400), (40, 12000, 528), (16, 16, 131056), (130, 17, 16400)]


@pytest.mark.parametrize("out,use_bias", [("fp16", False), ("bf16", True)])
@pytest.mark.parametrize("M,N,Kp", SHAPES)
def test_linear_codes(M, N, Kp, out, use_bias):
    X, W = _codes((M, Kp), M + N), _codes((N, Kp), N + Kp)
    g = torch.Generator().manual_seed(7)
    sx, sw = torch.rand(M, generator=g) * 2 / Kp ** 0.5, torch.rand(N, generator=g) * 1e-2
    bias = torch.randn(N, generator=g).to(DT[out]) if use_bias else None
    Y = fp6.int8_linear(X.to(DEV), W.to(DEV), sw.to(DEV), x_scales=sx.to(DEV),
                        bias=None if bias is None else bias.to(DEV), out_dtype=DT[out])
    ref, bound = int8_product(_f64(X), _f64(sx), _f64(W), _f64(sw), None if bias is None else _f64(bias), out)
    assert Y.shape == (M, N) and Y.dtype == DT[out]
    err = np.abs(_f64(Y) - ref)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("variant", range(1, 11))
@pytest.mark.parametrize("M,N,Kp", [(1, 1, 16), (1, 40, 2064), (17, 100, 64), (65, 31, 336), (130, 600, 4112),
                                    (257, 513, 2000), (300, 1032, 256), (513, 264, 128), (64, 64, 1024), (33, 72, 12304)])
def test_linear_every_variant(variant, M, N, Kp):
    # Scales are powers of two, so the only rounding is the last one: equal bits.
    X, W = _codes((M, Kp), M), _codes((N, Kp), N)
    bias = torch.randint(-8, 9, (N,), generator=torch.Generator().manual_seed(1)).half()
    Y = fp6.int8_linear_plan(X.to(DEV), W.to(DEV), torch.full((N,), 2.0 ** -8, device=DEV), torch.full((M,), 2.0 ** -4, device=DEV),
                             variant, bias=bias.to(DEV))
    p = X.double() @ W.double().t() * 2.0 ** -12
    exact = p.to(torch.float32).double() == p          # the sum fits fp32: no rounding before the bias
    assert exact.all()
    want = (p.float() + bias.float()).half()
    assert torch.equal(Y.cpu().view(torch.int16), want.view(torch.int16))


def test_linear_plan_refuses_unknown_variants():
    X, W = _codes((4, 64), 1).to(DEV), _codes((8, 64), 2).to(DEV)
    for v in (-1, 11):
        with pytest.raises(fp6.FP6Error, match="FP6_E_VALUE"):
            fp6.int8_linear_plan(X, W, torch.ones(8, device=DEV), torch.ones(4, device=DEV), v)


def test_linear_largest_sum():
    K = 131056
    X = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    W = torch.full((2, K), -128, dtype=torch.int8, device=DEV)
    W[1] = 127
    Y = fp6.int8_linear(X, W, torch.full((2,), 2.0 ** -20, device=DEV), x_scales=torch.ones(3, device=DEV))
    assert torch.equal(Y.double().cpu(), (torch.tensor([[16384.0 * K, -16256.0 * K]]) * 2.0 ** -20).half().double().expand(3, 2))


@pytest.mark.parametrize("M", [1, 2, 4, 5, 7, 16, 40, 150, 300])
@pytest.mark.parametrize("dtype,pad,K,N", [("fp16", 0, 1024, 512), ("bf16", 5, 1011, 77), ("fp16", 8, 333, 1000),
                                           ("fp16", 1, 8192, 40), ("bf16", 0, 4200, 33), ("fp16", 3, 1, 5),
                                           ("bf16", 0, 8208, 24)])
def test_linear_tokens_is_quantiser_then_product(M, dtype, pad, K, N):
    X = _tokens(M, K, dtype, M, pad)
    W, sw = fp6.int8_quantize_rows(np.random.default_rng(K).standard_normal((N, K)).astype(np.float32))
    W, sw = torch.from_numpy(W).to(DEV), torch.from_numpy(sw).to(DEV)
    bias = torch.randn(N, device=DEV).to(DT[dtype])
    Y = fp6.int8_linear(X, W, sw, bias=bias)
    q, s = fp6.int8_quantize_tokens(X)
    Y2 = fp6.int8_linear(q, W, sw, x_scales=s, bias=bias, out_dtype=DT[dtype])
    assert torch.equal(Y.view(torch.int16), Y2.view(torch.int16))
    qr, sr = int8_codes(_f64(X))
    ref, bound = int8_product(qr, sr, _f64(W)[:, :K], _f64(sw), _f64(bias), dtype)
    assert (np.abs(_f64(Y) - ref) <= bound).all()


def test_linear_tokens_zero_and_non_finite_rows():
    W, sw = _codes((40, 1008), 3).to(DEV), torch.rand(40, device=DEV)
    for M in (4, 9):
        X = _tokens(M, 1000, "fp16", M)
        X[1], X[2, 7], X[3, 999] = 0, float("nan"), float("-inf")
        y = fp6.int8_linear(X, W, sw)
        assert (y[1] == 0).all() and torch.isnan(y[2:4]).all() and torch.isfinite(y[0]).all()


def test_linear_near_the_true_product():
    # Codes of both sides are off by half a step of a/127 each; the sum of K such errors, as
    # independent uniform ones, stays within 6 of its standard deviations.
    M, N, K = 32, 64, 2048
    X, Wf = torch.randn(M, K, device=DEV).half(), torch.randn(N, K) * 0.05
    W, sw = fp6.int8_quantize_rows(Wf.numpy())
    Y = fp6.int8_linear(X, torch.from_numpy(W).to(DEV), torch.from_numpy(sw).to(DEV))
    x, w = _f64(X), Wf.double().numpy()
    sx = np.abs(x).max(1) / 127
    var = (sx[:, None] ** 2 * (w ** 2).sum(1)[None, :] + (x ** 2).sum(1)[:, None] * (sw.astype(np.float64) ** 2)[None, :]) / 12
    assert (np.abs(_f64(Y) - x @ w.T) <= 6 * np.sqrt(var) + 2.0 ** -11 * np.abs(x @ w.T) + 1e-6).all()


def test_linear_rows_behind_the_last_stay():
    X, W = _codes((5, 64), 1).to(DEV), _codes((9, 64), 2).to(DEV)
    buf = torch.full((8, 9), 3.0, dtype=torch.float16, device=DEV)
    fp6.int8_linear(X, W, torch.ones(9, device=DEV) * 1e-4, x_scales=torch.ones(5, device=DEV), out=buf[:5])
    assert (buf[5:] == 3).all()


def test_linear_empty_batch():
    Y = fp6.int8_linear(torch.empty(0, 20, dtype=torch.float16, device=DEV), _codes((4, 32), 1).to(DEV),
                        torch.ones(4, device=DEV))
    assert Y.shape == (0, 4)
    q, s = fp6.int8_quantize_tokens(torch.empty(0, 20, dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 32) and s.shape == (0,)


def test_linear_refuses_wrong_tensors():
    X, W, sw = _codes((4, 64), 1).to(DEV), _codes((8, 64), 2).to(DEV), torch.ones(8, device=DEV)
    sx = torch.ones(4, device=DEV)
    for kw in (dict(x_scales=sx[:3]), dict(x_scales=sx.double()), dict(x_scales=sx.cpu()),
               dict(x_scales=sx, bias=torch.ones(8, device=DEV)), dict(x_scales=sx, out_dtype=torch.float32),
               dict(x_scales=sx, out=torch.empty(4, 9, dtype=torch.float16, device=DEV)),
               dict(x_scales=sx, out=torch.empty(4, 8, dtype=torch.float16, device=DEV), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            fp6.int8_linear(X, W, sw, **kw)
    with pytest.raises(ValueError):
        fp6.int8_linear(X, W.t().contiguous().t(), sw, x_scales=sx)
    with pytest.raises(ValueError):
        fp6.int8_linear(torch.zeros(4, 65, dtype=torch.float16, device=DEV), W, sw)


def test_linear_other_stream_and_graph():
    X = _tokens(12, 1000, "fp16", 3)
    W, sw = _codes((300, 1008), 4).to(DEV), torch.rand(300, device=DEV) * 1e-3
    want = fp6.int8_linear(X, W, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fp6.int8_linear(X, W, sw, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp6.int8_linear(X, W, sw, out=out)
    for i in range(4):
        X.copy_(_tokens(12, 1000, "fp16", 10 + i))
        eager = fp6.int8_linear(X, W, sw)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
