"""Mixture-of-experts layer against 64-bit references (needs an MI355X)."""

import numpy as np
import pytest

import oracle

from _operators_ref import experts, int8_codes, int8_product, route

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import weight_only_fp6_amd as fp6  # noqa: E402

DEV = torch.device("cuda:0")
_cache = {}


class Dequantised:
    """The experts' matrices in float64, each made when it is asked for."""

    def __init__(self, codes, scales, fmt):
        self.codes, self.scales, self.fmt, self.shape = codes, scales, fmt, codes.shape

    def __getitem__(self, e):
        return oracle.dequant_ref(self.codes[e], self.scales[e], self.fmt).astype(np.float64)


class Experts:
    """A stack of random experts, packed on the GPU."""

    def __init__(self, E, H, I, fmt="e3m2", seed=0):
        rng = np.random.default_rng(seed + E + H + I)
        self.E, self.H, self.I, self.fmt = E, H, I, fmt
        self.args = []
        self.dq = []
        for rows, cols in ((2 * I, H), (H, I)):
            codes = rng.integers(0, 1 << fp6.bits(fmt), (E, rows, cols), dtype=np.uint8)
            top = {"e3m2": 28.0, "e2m3": 7.5, "e2m2": 7.0, "e2m1": 6.0}[fmt]
            scales = (rng.uniform(2, 4, (E, rows)) / top / cols ** 0.5).astype(np.float16)
            self.args += [torch.from_numpy(fp6.moe_prepack(codes, scales, fmt)).to(DEV), torch.from_numpy(scales).to(DEV)]
            self.dq.append(Dequantised(codes, scales, fmt))

    @classmethod
    def get(cls, *key):
        if key not in _cache:
            if len(_cache) > 3:
                _cache.clear()
            _cache[key] = cls(*key)
        return _cache[key]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _x(T, H, seed):
    return torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).half().to(DEV)


def _routing(T, E, k, seed, duplicates=False):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)) if duplicates else np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(T, k)
    w = rng.dirichlet(np.ones(k), T).astype(np.float32)
    return torch.from_numpy(ids.astype(np.int32)).to(DEV), torch.from_numpy(w).to(DEV)


def _check(y, ref, bound):
    got = _f64(y)
    err = np.abs(got - ref)
    assert (err <= bound).all(), (np.nanmax(err / bound), np.argwhere(~(err <= bound))[:4])


def _run(ex, X, ids, w):
    y = fp6.moe_experts(X, ids, w, *ex.args, fmt=ex.fmt)
    ref, bound = experts(_f64(X), ids.cpu().numpy(), _f64(w), *ex.dq)
    _check(y, ref, bound)
    return y


# --- experts ----------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e3m2", "e2m3", "e2m2", "e2m1"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 256), (3, 5, 3, 512, 768), (17, 4, 2, 1280, 256)])
def test_experts_formats(fmt, T, E, k, H, I):
    _run(Experts.get(E, H, I, fmt), _x(T, H, T), *_routing(T, E, k, T))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 6, 6), (15, 6, 2), (16, 6, 1), (18, 1, 1), (33, 6, 5), (50, 2, 2),
                                   (63, 6, 3), (64, 6, 4), (65, 6, 2), (130, 6, 1)])
def test_experts_tokens(T, E, k):
    ex = Experts.get(6, 512, 512)
    _run(ex, _x(T, 512, T), *_routing(T, E, k, T))


@pytest.mark.parametrize("H,I", [(256, 2304), (2304, 256), (4096, 512), (768, 4096), (8448, 256)])
def test_experts_sizes(H, I):
    ex = Experts.get(2, H, I)
    _run(ex, _x(3, H, 1), *_routing(3, 2, 1, 1))
    _run(ex, _x(20, H, 1), *_routing(20, 2, 2, 1))


def test_experts_many_and_top_k_16():
    ex = Experts.get(512, 256, 256, "e2m1")
    _run(ex, _x(2, 256, 1), *_routing(2, 512, 16, 1))
    _run(ex, _x(40, 256, 2), *_routing(40, 512, 16, 2))


@pytest.mark.parametrize("fmt", ["e3m2", "e2m3", "e2m2", "e2m1"])
@pytest.mark.parametrize("E,H,I", [(64, 512, 512), (128, 512, 512), (256, 512, 256), (128, 256, 1280)])
def test_experts_many_row_blocks(fmt, E, H, I):
    # The forms that share token fragments: every expert count per CU, up to 16 tokens and more.
    ex = Experts(E, H, I, fmt)
    _run(ex, _x(16, H, 1), *_routing(16, E, 16, 1))
    _run(ex, _x(20, H, 2), *_routing(20, E, 13, 2))


@pytest.mark.parametrize("fmt", ["e3m2", "e2m2", "e2m1"])
@pytest.mark.parametrize("H,I", [(256, 1280), (512, 1024), (768, 768), (1024, 512), (1280, 256), (2304, 256)])
def test_experts_shared_fragments_every_depth(H, I, fmt):
    # Fewer k-tiles than the ring of weights holds, whole turns of it and rests,
    # with one and two groups of columns and a second pass (expert 3 gets all).
    ex = Experts(128, H, I, fmt)
    for T in (16, 33, 64):
        ids, w = _routing(T, 128, 16, H + T)
        ids[:, 0] = 3
        _run(ex, _x(T, H, T + H), ids, w)


@pytest.mark.parametrize("E,H,I", [(64, 512, 512), (128, 512, 256), (6, 512, 512)])
def test_experts_uneven_routing(E, H, I):
    # One expert chosen by every token, one by 33, one by 32, one by 17, one by 16, the rest spread.
    ex = Experts.get(E, H, I)
    T, k = 64, 6
    rng = np.random.default_rng(5)
    ids = np.stack([np.concatenate([[3], rng.integers(0, E, k - 1)]) for _ in range(T)]).astype(np.int32)
    for j, (e, n) in enumerate([(1, 33), (0, 32), (4, 17), (5, 16)]):
        ids[:, 1 + j] = np.where(rng.permutation(T) < n, e, ids[:, 1 + j])
    w = rng.dirichlet(np.ones(k), T).astype(np.float32)
    _run(ex, _x(T, H, 1), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))


@pytest.mark.parametrize("E,T,k,H,I", [(6, 4, 2, 512, 512), (6, 16, 2, 256, 256), (40, 3, 3, 512, 256), (6, 33, 2, 512, 512),
                                       (128, 64, 16, 512, 256)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_experts_infinite_weights_stay_with_their_tokens(bad, E, T, k, H, I):
    # Expert 2 is unusable; tokens that did not choose it do not notice.
    ex = Experts(E, H, I)
    X = _x(T, H, 8)
    ids, w = _routing(T, E, k, 8)
    ids[ids == 2] = 3
    ref, bound = experts(_f64(X), ids.cpu().numpy(), _f64(w), *ex.dq)
    args = [t.clone() for t in ex.args]
    args[1][2] = bad
    args[3][2] = bad
    ids[1, k - 1] = 2
    y = fp6.moe_experts(X, ids, w, *args)
    others = np.arange(T) != 1
    _check(y[torch.from_numpy(others).to(DEV)], ref[others], bound[others])
    assert torch.isnan(y[1]).any()


def test_experts_same_index_twice():
    ex = Experts.get(6, 512, 512)
    for T, k in ((1, 4), (5, 6), (30, 8)):
        ids, w = _routing(T, 3, k, T, duplicates=True)
        _run(ex, _x(T, 512, T), ids, w)


@pytest.mark.parametrize("T", [1, 4, 40, 70])
def test_experts_not_served(T):
    ex = Experts.get(6, 512, 512)
    ids, w = _routing(T, 6, 3, T)
    for bad, row in ((-1, 0), (6, T // 2), (2 ** 31 - 1, T // 3), (-2 ** 31, T - 1)):
        ids[row, 1] = bad
        w[row, 1] = float("nan")          # of a choice that is not served: never read into a sum
    ids[T - 1] = -1
    wr = torch.where((ids < 0) | (ids >= 6), torch.zeros_like(w), w)
    X = _x(T, 512, T)
    y = fp6.moe_experts(X, ids, w, *ex.args)
    assert (y[T - 1] == 0).all()
    _check(y, *experts(_f64(X), ids.cpu().numpy(), _f64(wr), *ex.dq))
    assert (fp6.moe_experts(X, torch.full_like(ids, -1), w, *ex.args) == 0).all()


def test_experts_a_bad_token_stays_alone():
    ex = Experts.get(6, 512, 512)
    T = 21
    X, (ids, w) = _x(T, 512, 5), _routing(T, 6, 3, 5)
    clean = fp6.moe_experts(X, ids, w, *ex.args)
    Xb = X.clone()
    Xb[4, 7], Xb[9, 0] = float("nan"), float("inf")
    got = fp6.moe_experts(Xb, ids, w, *ex.args)
    keep = [t for t in range(T) if t not in (4, 9)]
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert torch.isnan(got[4]).any() and not torch.isfinite(got[9]).all()


def test_experts_large_gated_values():
    # |h| up to about 10^5: beyond fp16, inside what the layer carries.
    ex = Experts.get(2, 512, 256)
    X = _x(3, 512, 1) * 300
    ids, w = _routing(3, 2, 1, 1)
    g = np.stack([ex.dq[0][int(e)] @ x for e, x in zip(ids[:, 0].cpu(), _f64(X))])
    h = g[:, :256] / (1 + np.exp(-g[:, :256])) * g[:, 256:]
    assert 65504 < np.abs(h).max() < 2 ** 23
    w = w * 2.0 ** -8
    _run(ex, X, ids, w)
    w1 = torch.ones_like(w)
    y = fp6.moe_experts(X, ids, w1, *ex.args)
    ref, bound = experts(_f64(X), ids.cpu().numpy(), _f64(w1), *ex.dq)
    fits = np.abs(ref) + bound < 65504
    assert fits.any() and (np.abs(_f64(y) - ref) <= bound)[fits].all()


def test_experts_deterministic_and_workspace_contents_do_not_matter():
    ex = Experts.get(6, 512, 512)
    X, (ids, w) = _x(37, 512, 8), _routing(37, 6, 4, 8)
    want = fp6.moe_experts(X, ids, w, *ex.args)
    n = fp6.lib.fpx_moe_workspace_bytes(37, 6, 4, 512, 512)
    for fill in (0, 255, 0x7E):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        y = torch.empty_like(want)
        st = fp6.lib.fpx_moe_experts(0, X.data_ptr(), ids.data_ptr(), w.data_ptr(), *[a.data_ptr() for a in ex.args],
                                     y.data_ptr(), 37, 6, 4, 512, 512, ws.data_ptr(), n,
                                     torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(y, want)


def test_rows_behind_the_last_stay():
    ex = Experts.get(6, 512, 512)
    buf = torch.full((8, 512), 2.0, dtype=torch.float16, device=DEV)
    fp6.moe_experts(_x(5, 512, 1), *_routing(5, 6, 2, 1), *ex.args, out=buf[:5])
    assert (buf[5:] == 2).all()


# --- layer ------------------------------------------------------------------
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 6, 2), (4, 6, 6), (5, 6, 1), (16, 6, 3), (37, 6, 4), (66, 6, 2)])
def test_layer(T, E, k, renormalize):
    ex = Experts.get(6, 512, 512)
    X = _x(T, 512, T)
    router = (_x(E, 512, 99) * 0.1)
    y, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=k, renormalize=renormalize)
    rid, rw, rb = route(_f64(X), _f64(router), k, renormalize)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(_f64(w) - rw) <= rb).all()
    _check(y, *experts(_f64(X), rid, rw, *ex.dq, weight_bound=rb))
    y2 = fp6.moe_experts(X, ids, w, *ex.args)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("E,k", [(1, 1), (7, 7), (65, 3), (128, 5), (129, 5), (200, 16), (512, 8)])
def test_layer_many_experts(E, k):
    ex = Experts.get(E, 256, 256, "e2m1")
    for T in (1, 3, 4, 20):
        X, router = _x(T, 256, T), _x(E, 256, 7) * 0.2
        y, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=k, fmt="e2m1")
        rid, rw, rb = route(_f64(X), _f64(router), k, True)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert (np.abs(_f64(w) - rw) <= rb).all()
        _check(y, *experts(_f64(X), rid, rw, *ex.dq, weight_bound=rb))


@pytest.mark.parametrize("fmt", ["e3m2", "e2m3", "e2m2", "e2m1"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 2048, 256), (1, 9, 2, 2048, 256), (4, 4, 1, 1024, 256), (3, 5, 2, 1024, 256),
                                       (1, 64, 6, 256, 256), (1, 65, 6, 256, 256), (2, 4, 2, 256, 8192), (4, 17, 2, 256, 8192)])
def test_layer_small_router(T, E, k, H, I, fmt):
    """Both sides of the size up to which the first product takes the router
    itself, with few and many row blocks; equal router rows tie either way."""
    ex = Experts.get(E, H, I, fmt)
    X, router = _x(T, H, T), _x(E, H, 7) * (0.1 if H < 2048 else 0.03)
    router[E - 1] = router[0]
    y, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=k, fmt=fmt)
    rid, rw, rb = route(_f64(X), _f64(router), k, True)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(_f64(w) - rw) <= rb).all()
    _check(y, *experts(_f64(X), rid, rw, *ex.dq, weight_bound=rb))
    assert torch.equal(y, fp6.moe_experts(X, ids, w, *ex.args, fmt=fmt))


@pytest.mark.parametrize("T,E,k,H,I", [(5, 8, 2, 512, 256), (17, 128, 3, 512, 256), (16, 129, 3, 256, 256), (6, 16, 4, 4096, 256),
                                       (6, 17, 4, 4096, 256), (1024, 4, 2, 256, 256), (1025, 4, 2, 256, 256)])
def test_layer_choice_in_one_or_two_launches(T, E, k, H, I):
    """Both sides of the sizes up to which a token's logits and choice are one kernel."""
    ex = Experts.get(E, H, I, "e2m1")
    X, router = _x(T, H, T), _x(E, H, 7) * (0.1 if H < 2048 else 0.03)
    router[E - 1] = router[1]
    y, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=k, fmt="e2m1")
    rid, rw, rb = route(_f64(X), _f64(router), k, True)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(_f64(w) - rw) <= rb).all()
    _check(y, *experts(_f64(X), rid, rw, *ex.dq, weight_bound=rb))


def test_layer_ties_go_to_the_lower_index():
    ex = Experts.get(6, 512, 512)
    router = _x(6, 512, 3) * 0.1
    router[4] = router[1]
    router[5] = router[1]
    router[2] = 0
    router[3] = -router[2]                       # -0 ties with +0
    for T in (1, 9):
        X = _x(T, 512, T)
        _, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=6)
        rid, rw, _ = route(_f64(X), _f64(router), 6, True)
        assert np.array_equal(ids.cpu().numpy(), rid)
        for row, wr in zip(ids.tolist(), w.tolist()):
            i, j, l = row.index(1), row.index(4), row.index(5)
            assert j == i + 1 and l == j + 1 and wr[i] == wr[j] == wr[l]
            assert row.index(3) == row.index(2) + 1
    X = torch.zeros(2, 512, dtype=torch.float16, device=DEV)
    _, ids, w = fp6.moe_layer(X, router, *ex.args, top_k=4)
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and (w == 0.25).all()


def test_layer_near_ties_are_decided_in_64_bits():
    # Two experts whose logits differ by 2^-24 next to a sum of about 2^11: fp32 sums tie.
    ex = Experts.get(6, 512, 512)
    X = torch.full((3, 512), 2.0, dtype=torch.float16, device=DEV)
    router = torch.zeros(6, 512, dtype=torch.float16, device=DEV)
    router[0] = -1
    router[1:] = 2
    router[3, 11] = 2.0 + 2.0 ** -9
    X[:, 300], router[:, 300] = 2.0 ** -12, 0.0
    router[4, 300] = 2.0 ** -12
    _, ids, _ = fp6.moe_layer(X, router, *ex.args, top_k=4)
    assert ids.tolist() == [[3, 4, 1, 2]] * 3


def test_layer_not_a_number():
    ex = Experts.get(6, 512, 512)
    X, router = _x(6, 512, 1), _x(6, 512, 2) * 0.1
    want = fp6.moe_layer(X, router, *ex.args, top_k=2)
    Xb = X.clone()
    Xb[3, 100] = float("nan")
    got = fp6.moe_layer(Xb, router, *ex.args, top_k=2)
    assert got[1][3].tolist() == [0, 1] and torch.isnan(got[2][3]).all() and torch.isnan(got[0][3]).all()
    keep = [0, 1, 2, 4, 5]
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep])


def test_layer_empty_batch_and_refusals():
    ex = Experts.get(6, 512, 512)
    router = _x(6, 512, 2)
    y, ids, w = fp6.moe_layer(_x(0, 512, 1), router, *ex.args, top_k=2)
    assert y.shape == (0, 512) and ids.shape == (0, 2) and w.shape == (0, 2)
    X = _x(2, 512, 1)
    for bad in (0, 7):
        with pytest.raises(ValueError):
            fp6.moe_layer(X, router, *ex.args, top_k=bad)
    with pytest.raises(ValueError):
        fp6.moe_layer(X, router[:5], *ex.args, top_k=2)
    with pytest.raises(ValueError):
        fp6.moe_layer(X, router, *ex.args, top_k=2, fmt="e2m1")
    with pytest.raises(ValueError):
        fp6.moe_layer(X.float(), router, *ex.args, top_k=2)
    ids, w = _routing(2, 6, 2, 1)
    for bad in (ids.long(), ids[:1], ids.cpu()):
        with pytest.raises(ValueError):
            fp6.moe_experts(X, bad, w, *ex.args)
    with pytest.raises(ValueError):
        fp6.moe_experts(X, ids, w.half(), *ex.args)


# --- streams and graphs -----------------------------------------------------
def test_two_streams_at_once():
    ex = Experts.get(6, 512, 512)
    router = _x(6, 512, 2) * 0.1
    Xs = [_x(t, 512, t) for t in (3, 40)]
    want = [fp6.moe_layer(X, router, *ex.args, top_k=3) for X in Xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(fp6.moe_layer(Xs[i], router, *ex.args, top_k=3, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for res in got[i]:
            for a, b in zip(res, want[i]):
                assert torch.equal(a, b)


def test_two_graphs_and_eager_calls():
    ex = Experts.get(6, 512, 512)
    router = _x(6, 512, 2) * 0.1
    Xs = [_x(t, 512, t) for t in (1, 35)]
    fp6.moe_layer(Xs[0], router, *ex.args, top_k=3)
    graphs, outs = [], []
    for X in Xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fp6.moe_layer(X, router, *ex.args, top_k=3))
        graphs.append(g)
    for i in range(4):
        for X in Xs:
            X.copy_(_x(X.shape[0], 512, 50 + i))
        want = [fp6.moe_layer(X, router, *ex.args, top_k=3) for X in Xs]
        for res in outs:
            res[0].zero_()
        for g in graphs:
            g.replay()
        fp6.moe_layer(Xs[1], router, *ex.args, top_k=1)
        torch.cuda.synchronize()
        for res, ref in zip(outs, want):
            for a, b in zip(res, ref):
                assert torch.equal(a, b)


# --- a decoder block's linear work: W8A8 projection, then the experts ---------
@pytest.mark.parametrize("T", [1, 6, 48])
def test_projection_then_experts(T):
    H, I, E, k = 512, 512, 6, 2
    ex = Experts.get(E, H, I)
    rng = np.random.default_rng(T)
    W, sw = fp6.int8_quantize_rows((rng.standard_normal((H, H)) / H ** 0.5).astype(np.float32))
    W, sw = torch.from_numpy(W).to(DEV), torch.from_numpy(sw).to(DEV)
    router = _x(E, H, 2) * 0.1
    attn, resid = _x(T, H, T + 1), _x(T, H, T + 2)

    def block():
        o = fp6.int8_linear(attn, W, sw)
        x = resid + o
        y, ids, w = fp6.moe_layer(x, router, *ex.args, top_k=k)
        return o, x, ids, w, y, x + y

    out = block()
    o, x, ids, w, y, _ = out
    q, s = int8_codes(_f64(attn))
    ref, bound = int8_product(q, s, _f64(W), _f64(sw), None, "fp16")
    _check(o, ref, bound)
    rid, rw, rb = route(_f64(x), _f64(router), k, True)
    assert np.array_equal(ids.cpu().numpy(), rid) and (np.abs(_f64(w) - rw) <= rb).all()
    _check(y, *experts(_f64(x), rid, rw, *ex.dq, weight_bound=rb))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rep = block()
    for i in range(3):
        attn.copy_(_x(T, H, 70 + i))
        want = block()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(rep, want):
            assert torch.equal(a, b)
