"""Plain 64-bit references and error bounds of the int8 linear layer and the
mixture-of-experts layer, shared by their tests (NumPy only)."""

import numpy as np

HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}    # one rounding, relative
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}       # half a subnormal step
U32 = 2.0 ** -24


def int8_codes(x):
    """(codes float64 [M,K], scales float64 [M]) of finite rows: RNE(127 x / a), a / 127.

    The quotient of values of at most 24 bits is either exactly halfway or at least
    2^-32 of itself away from halfway, so its rounding to 53 bits decides correctly."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(axis=1)
    safe = np.where(a > 0, a, 1.0)
    return np.rint(127.0 * x / safe[:, None]), (a / 127.0).astype(np.float32).astype(np.float64)


def int8_product(q, sx, w, sw, bias, out):
    """(Y, bound): the sum of codes is exact (below 2^53); the kernel converts it to fp32,
    multiplies twice and adds the bias -- at most 4 roundings of 2^-24 of |product| + |bias| --
    and rounds once to the output type."""
    p = (q @ w.T) * sw[None, :] * sx[:, None]
    b = 0.0 if bias is None else bias[None, :]
    y = p + b
    slack = 4 * U32 * (np.abs(p) + np.abs(b)) * 1.01
    return y, slack + HALF_STEP[out] * (np.abs(y) + slack) + TINY[out]


def route(x, router, k, renormalize):
    """(ids, weights, bound of the weights).

    Differences l - max are rounded to fp32 (2^-24 of themselves, which exp turns into as much
    of the weight), exp is good to 2 steps, the sum has at most E/64 + 6 (or k) additions and the
    quotient one rounding: (2 * (|l - max| + 3) + E/64 + k + 8) * 2^-24 of the weight."""
    logits = x @ router.T
    key = np.where(np.isnan(logits), np.inf, logits)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    best = np.take_along_axis(logits, ids, 1)
    top = best[:, :1]
    e = np.exp(best - top)
    w = e / (e.sum(1, keepdims=True) if renormalize else np.exp(logits - top).sum(1, keepdims=True))
    span = np.abs(logits - top).max(axis=1, keepdims=True)
    return ids, w, w * (2 * (span + 3) + router.shape[0] / 64 + k + 8) * U32


def experts(x, ids, weights, w13, w2, weight_bound=None):
    """(Y, bound) of the experts.

    With u = 2^-24 and sums of n products in any order off by at most n u times the sum of
    magnitudes: gate and up by H u sum|x w|; silu has slope below 1.1 and its exp, sum and
    quotient cost 8 u; h is carried in 22 bits, or to 2^-28 where it is small (2^-8 * 2^-24
    in the low half's 2^-11 steps is finer); the second product adds I * (choices) terms plus
    the 64 partial sums of waves and experts; Y is rounded once."""
    T, H = x.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    y, slack = np.zeros((T, H)), np.zeros((T, H))
    many = [len({int(e) for e in ids[t] if 0 <= e < E}) for t in range(T)]
    for e in sorted({int(e) for e in np.asarray(ids).ravel() if 0 <= e < E}):
        up, down = w13[e], w2[e]
        aup, adown = np.abs(up), np.abs(down)
        for t in range(T):
            hit = [j for j in range(ids.shape[1]) if ids[t, j] == e]
            if not hit:
                continue
            wt = weights[t, hit].sum()
            dw = len(hit) * U32 * np.abs(weights[t, hit]).sum()
            if weight_bound is not None:
                dw += weight_bound[t, hit].sum()
            gu = up @ x[t]
            d = H * U32 * (aup @ np.abs(x[t]))
            g, u, dg, du = gu[:I], gu[I:], d[:I], d[I:]
            act = g / (1 + np.exp(-g))
            h = act * u * wt
            dh = ((1.1 * dg + 8 * U32 * np.abs(act)) * (np.abs(u) + du) + np.abs(act) * du) * (abs(wt) + dw)
            dh += np.abs(act * u) * dw + (4 * U32 + 2.0 ** -22) * np.abs(h) + 2.0 ** -28
            y[t] += down @ h
            n = I * many[t] + 64
            slack[t] += adown @ dh + n * U32 * (adown @ (np.abs(h) + dh))
    return y, slack + HALF_STEP["fp16"] * (np.abs(y) + slack) + TINY["fp16"]
