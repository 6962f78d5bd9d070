"""Measured cases of the W8A8 linear layer and the mixture-of-experts layer.

Operators:

* ``int8_quantize_tokens`` -- 8-bit codes and one scale for each token;
* ``int8_linear`` -- product of 8-bit integers with a scale for each token and channel;
* ``moe_layer`` -- router, top-k choice and gated experts in FPx weights, for few tokens;
* ``moe_experts`` -- the experts alone, for routing that the caller brings.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, through the library's entry points.
"""

import math

import torch

own = False

# Exponent and mantissa bits, exponent bias and largest magnitude of the weight formats.
FORMATS = {"e3m2": (3, 2, 3, 28.0), "e2m3": (2, 3, 1, 7.5), "e2m2": (2, 2, 1, 7.0), "e2m1": (2, 1, 1, 6.0)}
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One decode step's batch of hidden states, quantised once for q, k and v.
        {"name": "quantize_16x4096", "op": "quantize", "M": 16, "K": 4096, "dtype": "fp16", "strided": False},
        # The hidden states of a long prompt.
        {"name": "quantize_4096x8192_bf16", "op": "quantize", "M": 4096, "K": 8192, "dtype": "bf16", "strided": False},
        # Attention projection of a 7B layer for one token: latency counts.
        {"name": "int8_1x4096x4096", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "fp16",
         "quantized": False, "bias": False, "strided": False},
        # MLP of a 70B layer for a decode batch: the weights' bytes count.
        {"name": "int8_16x28672x8192", "op": "linear", "M": 16, "N": 28672, "K": 8192, "dtype": "fp16",
         "quantized": False, "bias": False, "strided": False},
        # QKV projection of a 30B layer for a short prompt, codes made before.
        {"name": "int8_128x21504x7168", "op": "linear", "M": 128, "N": 21504, "K": 7168, "dtype": "fp16",
         "quantized": True, "bias": True, "strided": False},
        # A ragged prompt and layer: no size is a multiple of a tile, rows are a part of wider ones.
        {"name": "int8_333x5003x2011_bf16", "op": "linear", "M": 333, "N": 5003, "K": 2011, "dtype": "bf16",
         "quantized": False, "bias": True, "strided": True},
        # MLP of a 7B layer over a long prompt: the product itself counts.
        {"name": "int8_4096x11008x4096", "op": "linear", "M": 4096, "N": 11008, "K": 4096, "dtype": "fp16",
         "quantized": True, "bias": False, "strided": False},
        # A small layer for one token: launches and latency count.
        {"name": "moe_1_e8k2_1024x512", "op": "layer", "T": 1, "E": 8, "k": 2, "H": 1024, "I": 512,
         "fmt": "e3m2", "renormalize": True},
        # One token of a layer with many narrow experts.
        {"name": "moe_1_e64k8_2048x1024", "op": "layer", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1024,
         "fmt": "e3m2", "renormalize": True},
        # A decode batch of a layer with wide experts, nearly all of them used.
        {"name": "moe_16_e16k4_4096x2048_e2m1", "op": "layer", "T": 16, "E": 16, "k": 4, "H": 4096, "I": 2048,
         "fmt": "e2m1", "renormalize": False},
        # A shard's part of a routed batch: some choices and the last rows are not its own.
        {"name": "experts_7_e40k3_1280x768_e2m3", "op": "experts", "T": 7, "E": 40, "k": 3, "H": 1280, "I": 768,
         "fmt": "e2m3", "masked": True},
        # The largest batch that still counts as few tokens: every expert's weights are read once.
        {"name": "experts_64_e64k8_2048x1024", "op": "experts", "T": 64, "E": 64, "k": 8, "H": 2048, "I": 1024,
         "fmt": "e3m2", "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "layer", "layer", "experts"])
    if op == "quantize":
        K = _log(rng, 32, 8192)
        return {"op": op, "M": _log(rng, 1, min(8192, (1 << 25) // K)), "K": K,
                "dtype": rng.choice(sorted(DTYPES)), "strided": rng.random() < 0.3}
    if op == "linear":
        N, K = _log(rng, 64, 16384), _log(rng, 64, 8192)
        M = _log(rng, 1, max(1, min(4096, (4096 * 11008 * 4096) // (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(sorted(DTYPES)),
                "quantized": rng.random() < 0.4, "bias": rng.random() < 0.5, "strided": rng.random() < 0.3}
    H, I = 256 * _log(rng, 2, 16), 256 * _log(rng, 1, 8)
    E = _log(rng, 4, max(4, min(96, (64 * 2048 * 1024) // (H * I))))
    c = {"op": op, "T": _log(rng, 1, 64), "E": E, "k": rng.randint(1, min(8, E)), "H": H, "I": I,
         "fmt": rng.choice(sorted(FORMATS))}
    c["renormalize" if op == "layer" else "masked"] = rng.random() < 0.5
    return c


def _padded(K):
    return (K + 15) // 16 * 16


def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def _tokens(case, gen, rows, cols):
    x = _normal((rows, cols + (37 if case.get("strided") else 0)), gen)
    x[:, :: max(1, cols // 7)] *= 8.0  # a few channels far larger than the others, as hidden states have
    return x.to(DTYPES[case.get("dtype", "fp16")])[:, :cols]


def _int8_rows(w, K):
    """Codes of fp32 rows, padded with zeros, and their scales."""
    top = w.abs().amax(1)
    q = torch.zeros((w.shape[0], _padded(K)), dtype=torch.int8, device=w.device)
    q[:, :K] = torch.round(w * (127.0 / top)[:, None]).to(torch.int8)
    return q, top / 127.0


def _fpx_rows(w, fmt):
    """The format's codes of fp32 rows, nearest magnitude, and their fp16 scales."""
    table = _values(fmt, w.device)
    half = table.shape[0] // 2
    s = (w.abs().amax(1) / FORMATS[fmt][3]).half()
    mag = torch.bucketize(w.abs() / s.float()[:, None], (table[1:half] + table[: half - 1]) / 2)
    return (mag + half * (w < 0)).to(torch.uint8), s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "quantize":
        return {"case": case, "X": _tokens(case, gen, case["M"], case["K"])}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st = {"case": case, "X": _tokens(case, gen, M, K)}
        st["W"], st["w_scales"] = _int8_rows(_normal((N, K), gen, K ** -0.5), K)
        st["bias"] = _normal((N,), gen, 0.1).to(DTYPES[case["dtype"]]) if case["bias"] else None
        st["x_scales"] = None
        if case["quantized"]:
            st["X"], st["x_scales"] = _int8_rows(st["X"].float(), K)
        return st
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    st = {"case": case, "X": _normal((T, H), gen).half()}
    if case["op"] == "layer":
        st["router"] = _normal((E, H), gen, H ** -0.5).half()
    else:
        st["ids"] = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].int().contiguous()
        st["weights"] = torch.softmax(_normal((T, k), gen), 1)
        if case["masked"]:
            st["ids"].masked_fill_(torch.rand((T, k), generator=gen, device="cuda") < 0.25, -1)
            st["ids"][T - T // 4:] = -1
    for name, rows, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        codes = torch.empty((E, rows, cols), dtype=torch.uint8, device="cuda")
        scales = torch.empty((E, rows), dtype=torch.float16, device="cuda")
        for e in range(E):
            codes[e], scales[e] = _fpx_rows(_normal((rows, cols), gen, cols ** -0.5), case["fmt"])
        st[name], st[name + "_scales"] = codes, scales
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and "down" in st:  # a program packs its weights once, when it loads them
        import weight_only_fp6_amd as fp6
        for name in ("gate_up", "down"):
            packed = fp6.moe_prepack(st[name].cpu().numpy(), st[name + "_scales"].cpu().numpy(), case["fmt"])
            st[name] = torch.from_numpy(packed).cuda()
    return st


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _values(fmt, device):
    """Every code's value: sign on top, subnormals, no infinities."""
    e_bits, m_bits, bias, _ = FORMATS[fmt]
    c = torch.arange(1 << (e_bits + m_bits), device=device)
    e, m = c >> m_bits, (c & ((1 << m_bits) - 1)).float() / (1 << m_bits)
    mag = torch.where(e > 0, (1 + m) * torch.exp2((e - bias).float()), m * 2.0 ** (1 - bias))
    return torch.cat([mag, -mag])


def _plain_quantize(X):
    x = X.float()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    return q, top[:, 0] / 127.0


def _plain_linear(st):
    K = st["case"]["K"]
    if st["x_scales"] is None:
        q, s = _plain_quantize(st["X"])
    else:
        q, s = st["X"][:, :K].float(), st["x_scales"]
    y = torch.matmul(q, st["W"][:, :K].float().t()) * st["w_scales"] * s[:, None]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(DTYPES[st["case"]["dtype"]])


def _plain_route(st):
    c = st["case"]
    logits = torch.matmul(st["X"].double(), st["router"].double().t())
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp(best - best[:, :1])
    w = p[:, : c["k"]] / (p[:, : c["k"]].sum(1, keepdim=True) if c["renormalize"] else p.sum(1, keepdim=True))
    return ids[:, : c["k"]].int(), w.float()


def _plain_weights(codes, scales, fmt):
    return (_values(fmt, codes.device)[codes.int()] * scales.float()[..., None]).half().float()


def _plain_experts(st, ids, weights):
    c = st["case"]
    t, j = torch.nonzero((ids >= 0) & (ids < c["E"]), as_tuple=True)
    used, at = torch.unique(ids[t, j], return_inverse=True)  # the experts that any token chose
    share = torch.zeros((c["T"], used.numel()), device=ids.device)
    share.index_put_((t, at), weights[t, j], accumulate=True)
    up = _plain_weights(st["gate_up"][used], st["gate_up_scales"][used], c["fmt"])
    gu = torch.matmul(st["X"].float(), up.transpose(1, 2))  # [used, T, 2I]
    g, u = gu[..., : c["I"]], gu[..., c["I"]:]
    h = g / (1 + torch.exp(-g)) * u * share.t()[..., None]
    down = _plain_weights(st["down"][used], st["down_scales"][used], c["fmt"])
    return torch.matmul(h, down.transpose(1, 2)).sum(0).half()


def run(state):
    c = state["case"]
    if own:
        import weight_only_fp6_amd as fp6
        if c["op"] == "quantize":
            q, s = fp6.int8_quantize_tokens(state["X"])
            return {"values": q[:, : c["K"]] * s[:, None], "scales": s}
        if c["op"] == "linear":
            return fp6.int8_linear(state["X"], state["W"], state["w_scales"], x_scales=state["x_scales"],
                                   bias=state["bias"], out_dtype=DTYPES[c["dtype"]])
        experts = (state["gate_up"], state["gate_up_scales"], state["down"], state["down_scales"])
        if c["op"] == "layer":
            y, ids, w = fp6.moe_layer(state["X"], state["router"], *experts, top_k=c["k"],
                                      renormalize=c["renormalize"], fmt=c["fmt"])
            return {"y": y, "ids": ids, "weights": w}
        return {"y": fp6.moe_experts(state["X"], state["ids"], state["weights"], *experts, fmt=c["fmt"])}
    if c["op"] == "quantize":
        q, s = _plain_quantize(state["X"])
        return {"values": q * s[:, None], "scales": s}
    if c["op"] == "linear":
        return _plain_linear(state)
    if c["op"] == "layer":
        ids, w = _plain_route(state)
        return {"y": _plain_experts(state, ids, w), "ids": ids, "weights": w}
    return {"y": _plain_experts(state, state["ids"], state["weights"])}


def work(case):
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        # values come back, not codes: four bytes for each
        return {"bytes": 2 * M * K + 4 * M * K + 4 * M, "flops": 3 * M * K}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K + (1 if case["quantized"] else 2) * M * K + 2 * M * N + 4 * N
                + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    bits = 1 + sum(FORMATS[case["fmt"]][:2])
    pairs = T * k
    if case.get("masked"):
        pairs = 0.75 * k * (T - T // 4)
    used = E * (1 - (1 - 1 / E) ** pairs) if case["op"] == "experts" else E * (1 - (1 - k / E) ** T)
    b = used * 3 * H * I * bits / 8 + 4 * T * H + 8 * T * k
    f = 6 * H * I * pairs
    if case["op"] == "layer":
        b, f = b + 2 * E * H, f + 2 * T * E * H
    return {"bytes": int(b), "flops": int(f)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _exact_codes(X):
    x = X.double()
    top = x.abs().max(dim=1).values
    return torch.round(127 * x / top.clamp_min(1e-300)[:, None]), top / 127


def _exact_matrix(codes, scales, fmt):
    """fp16(value * scale) of one expert's codes, by the format's fields."""
    e_bits, m_bits, bias, _ = FORMATS[fmt]
    c = codes.to(torch.int32)
    m, e, sign = c % (1 << m_bits), (c >> m_bits) % (1 << e_bits), c >> (e_bits + m_bits)
    frac = m + torch.where(e > 0, 1 << m_bits, 0)
    v = torch.ldexp(frac.double(), torch.clamp_min(e, 1) - bias - m_bits) * (1 - 2 * sign)
    return (v * scales.double()[:, None]).to(torch.float16).double()


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "quantize":
        q, s = _exact_codes(st["X"])
        return {"values": q * s.float().double()[:, None], "scales": s}
    if case["op"] == "linear":
        K = case["K"]
        q, s = (st["X"][:, :K].double(), st["x_scales"].double()) if case["quantized"] else _exact_codes(st["X"])
        y = (q @ st["W"][:, :K].double().T) * torch.outer(s, st["w_scales"].double())
        return y if st["bias"] is None else y + st["bias"].double()
    x, T, E, k, I = st["X"].double(), case["T"], case["E"], case["k"], case["I"]
    out = {}
    if case["op"] == "layer":
        logits = x @ st["router"].double().T
        ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
        w = torch.softmax(logits, 1).gather(1, ids)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        out = {"ids": ids.int(), "weights": w}
    else:
        ids, w = st["ids"].long(), st["weights"].double()
    y = torch.zeros((T, case["H"]), dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gu = x[t] @ _exact_matrix(st["gate_up"][e], st["gate_up_scales"][e], case["fmt"]).T
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:] * w[t, j][:, None]
            y.index_add_(0, t, h @ _exact_matrix(st["down"][e], st["down_scales"][e], case["fmt"]).T)
    return {"y": y, **out}
