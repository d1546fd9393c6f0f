"""Cases that measure the microscaled 4-bit operators and the whole mixture-of-experts layer.

Five operators, each computed in two ways on the same inputs: through the
framework's calls where `own` is true, and otherwise in elementary torch
operations, in 32 bits (the router in 64: the choice of experts goes by values
that may lie next to each other).

  quantise   kq_mx4_quantize, kq_mx4_dequantize: blocks of 32 values of a row
             share one power-of-two scale (a byte, biased by 127) and keep four
             bits each (sign, two exponent bits, one mantissa bit)
  gemv       kq_mx4_gemv: microscaled weights times a few activation columns
             held in 16 or 32 bits (decode, verify)
  gemm       kq_mx4_gemm: microscaled weights times microscaled activations
             (prompts)
  route      kq_moe_route: router product, softmax and choice of the best
             top_k experts of each token
  moe        kq_mx4_moe_layer: the router and the chosen experts' gated FFN
             with microscaled weights, summed with the router's weights

A microscaled matrix is two planes: codes uint8 [R][K/2] (element 2i in the
low nibble of byte i) and scales uint8 [R][K/32].
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
#: The eight magnitudes of a code's low three bits; bit 3 is the sign.
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # Activations of a verify pass of 16 rows, hidden size 2560: the call whose launch counts.
        {"name": "quantise_16x2560_bf16", "op": "quantise", "R": 16, "K": 2560, "type": "bf16"},
        # Activations of a ragged prompt going into a 9728-wide down projection.
        {"name": "quantise_1111x9728_f16", "op": "quantise", "R": 1111, "K": 9728, "type": "f16"},
        # The gate and up weights of one layer, quantised from 32 bits when a model is loaded.
        {"name": "quantise_19456x2560_f32", "op": "quantise", "R": 19456, "K": 2560, "type": "f32"},
        # One decode token through the gate and up projection of the 4B-shaped stack.
        {"name": "gemv_19456x2560_m1_bf16", "op": "gemv", "N": 19456, "K": 2560, "M": 1, "type": "bf16"},
        # A verify pass of eight rows through the query, key and value projection.
        {"name": "gemv_6144x2560_m8_f16", "op": "gemv", "N": 6144, "K": 2560, "M": 8, "type": "f16"},
        # Three requests of 16 rows each sharing one pass over the down projection.
        {"name": "gemv_2560x9728_m48_bf16", "op": "gemv", "N": 2560, "K": 9728, "M": 48, "type": "bf16"},
        # A short ragged prompt through a matrix of odd sizes, kept in 32 bits.
        {"name": "gemm_77x1000x1056_f32", "op": "gemm", "M": 77, "N": 1000, "K": 1056, "type": "f32"},
        # A long prompt through the down projection.
        {"name": "gemm_4096x2560x9728_bf16", "op": "gemm", "M": 4096, "N": 2560, "K": 9728, "type": "bf16"},
        # The router of one decode token: 128 experts, the best eight.
        {"name": "route_m1_e128_k8_f16", "op": "route", "M": 1, "K": 2048, "E": 128, "top_k": 8, "type": "f16", "renorm": True},
        # The router of a shared pass of 48 rows over 512 experts, the best ten, weights of all experts' softmax.
        {"name": "route_m48_e512_k10_bf16", "op": "route", "M": 48, "K": 2048, "E": 512, "top_k": 10, "type": "bf16", "renorm": False},
        # One decode token through the layer of 128 experts (hidden 2048, FFN 768, the best eight).
        {"name": "moe_m1_e128_k8_f16", "op": "moe", "M": 1, "K": 2048, "I": 768, "E": 128, "top_k": 8, "type": "f16", "renorm": True},
        # A verify pass of 16 rows through the same layer: most experts serve one or two rows.
        {"name": "moe_m16_e128_k8_bf16", "op": "moe", "M": 16, "K": 2048, "I": 768, "E": 128, "top_k": 8, "type": "bf16", "renorm": True},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(step, min(high // step, max(1, round(v / step))) * step)


def draw(rng):
    op = rng.choice(["quantise", "gemv", "gemv", "gemm", "route", "moe", "moe"])
    kind = rng.choice(["f32", "f16", "bf16"])
    while True:
        if op == "quantise":
            c = {"op": op, "R": _log(rng, 1, 20000), "K": _log(rng, 32, 16384, 32), "type": kind}
            if c["R"] * c["K"] <= 19456 * 2560:
                return c
        elif op == "gemv":
            c = {"op": op, "N": _log(rng, 16, 20000), "K": _log(rng, 32, 16384, 32), "M": rng.randint(1, 64), "type": kind}
            if c["N"] * c["K"] <= 19456 * 2560:
                return c
        elif op == "gemm":
            c = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 16, 20000), "K": _log(rng, 32, 16384, 32), "type": kind}
            if c["M"] * c["N"] * c["K"] <= 4096 * 2560 * 9728 and (c["M"] + c["N"]) * c["K"] <= 19456 * 2560:
                return c
        elif op == "route":
            c = {"op": op, "M": rng.randint(1, 64), "K": _log(rng, 64, 8192, 32), "E": _log(rng, 4, 512), "type": kind, "renorm": rng.random() < 0.5}
            c["top_k"] = rng.randint(1, min(16, c["E"]))
            return c
        else:
            c = {"op": op, "M": _log(rng, 1, 64), "K": _log(rng, 64, 4096, 32), "I": _log(rng, 32, 2048, 32), "E": _log(rng, 4, 256), "type": kind, "renorm": rng.random() < 0.5}
            c["top_k"] = rng.randint(1, min(12, c["E"]))
            if min(c["E"], c["M"] * c["top_k"]) * c["K"] * c["I"] <= 128 * 2048 * 768 and c["E"] * c["K"] * c["I"] <= 256 * 2048 * 768:
                return c


def _shift(x, n):
    """x times 2 to the whole numbers n (-127 to 127), exactly."""
    return torch.ldexp(x, n)


def _exponent(amax):
    """The block exponent: floor(log2(amax)) - 2, so that the largest value of
    a block lands in [4, 8), within what a scale byte holds; zero blocks take
    the least."""
    e = torch.frexp(amax)[1].to(torch.int32) - 3
    return torch.where(amax == 0, -127, e).clamp(-127, 127)


def _encode(x):
    """Codes uint8 [R][K/2] and scales uint8 [R][K/32] of x [R][K], in 32 bits:
    the nearest code, the even one on ties, 6 where a value is larger."""
    v = x.float().reshape(x.shape[0], -1, 32)
    e = _exponent(v.abs().amax(-1))
    a = _shift(v.abs(), -e[..., None])
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(x.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _decode(codes, scales, dtype=torch.float32):
    """The values of a microscaled matrix (any leading axes)."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).to(torch.int32)
    v = table[both].reshape(*scales.shape, 32)
    v = v * torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), scales.to(torch.int32) - 127)[..., None]
    return v.flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def weights(*shape):
        """A microscaled matrix of N(0, 0.02) weights, as a loaded model holds it."""
        codes, scales = _encode(normal(math.prod(shape[:-1]), shape[-1]) * 0.02)
        return codes.reshape(*shape[:-1], -1), scales.reshape(*shape[:-1], -1)

    def activations(rows, k):
        """Rows of a hidden state: a few channels are far larger than the others."""
        return normal(rows, k) * torch.exp(0.5 * normal(k))

    s = {"case": case}
    op, M, K = case["op"], case.get("M"), case["K"]
    if op == "quantise":
        R = case["R"]
        s["x"] = (activations(R, K) if case["type"] != "f32" else normal(R, K) * 0.02).to(dtype)
        s["codes"] = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(R, K // 32, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    elif op == "gemv":
        s["x"] = activations(M, K).to(dtype)
        s["w"] = weights(case["N"], K)
        s["y"] = torch.empty(M, case["N"], device="cuda")
    elif op == "gemm":
        s["a"] = _encode(activations(M, K))
        s["w"] = weights(case["N"], K)
        s["y"] = torch.empty(M, case["N"], dtype=dtype, device="cuda")
    else:
        E, top_k = case["E"], case["top_k"]
        s["x"] = normal(M, K).to(dtype)
        s["router"] = (normal(E, K) * K ** -0.5).to(dtype)
        s["ids"] = torch.empty(M, top_k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(M, top_k, device="cuda")
        if op == "moe":
            s["gate"], s["up"] = weights(E, case["I"], K), weights(E, case["I"], K)
            s["down"] = weights(E, K, case["I"])
            s["y"] = torch.empty(M, K, device="cuda")
    return s


def _own(s):
    import block_quantized_gemv_kq_amd as kq

    c = s["case"]
    op, M, K, kind = c["op"], c.get("M"), c["K"], c["type"]
    if op == "quantise":
        kq.kq_mx4_quantize(kind, s["x"], K, s["codes"], s["scales"], c["R"], K)
        kq.kq_mx4_dequantize(s["codes"], s["scales"], "bf16", s["values"], K, c["R"], K)
        return s["values"]
    if op == "gemv":
        kq.kq_mx4_gemv(*s["w"], kind, s["x"], s["y"], c["N"], K, M)
        return s["y"]
    if op == "gemm":
        kq.kq_mx4_gemm(*s["a"], *s["w"], kind, s["y"], M, c["N"], K)
        return s["y"]
    E, top_k = c["E"], c["top_k"]
    if "workspace" not in s:   # a program keeps its workspace from call to call
        n = kq.kq_moe_route_workspace_bytes(M, E) if op == "route" else kq.kq_mx4_moe_layer_workspace_bytes(K, c["I"], M, top_k, E)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    ws = s["workspace"]
    if op == "route":
        kq.kq_moe_route(kind, s["x"], kind, s["router"], M, K, E, top_k, c["renorm"], s["ids"], s["weights"], ws, ws.numel())
        return s["ids"], s["weights"]
    kq.kq_mx4_moe_layer(kind, s["x"], kind, s["router"], *s["gate"], *s["up"], *s["down"], s["y"], s["ids"], s["weights"],
                        K, c["I"], M, top_k, E, c["renorm"], ws, ws.numel())
    return s["y"], s["ids"], s["weights"]


def _route(s):
    """ids [M][top_k] (the largest logit first, the lowest index on ties) and their softmax weights, in 64 bits."""
    logits = s["x"].double() @ s["router"].double().T
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    p = torch.exp(best - best[:, :1])
    k = s["case"]["top_k"]
    total = (p[:, :k] if s["case"]["renorm"] else p).sum(-1, keepdim=True)
    return ids[:, :k], p[:, :k] / total


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    op = c["op"]
    if op == "quantise":
        return _decode(*_encode(state["x"])).bfloat16()
    if op == "gemv":
        return state["x"].float() @ _decode(*state["w"]).T
    if op == "gemm":
        return (_decode(*state["a"]) @ _decode(*state["w"]).T).to(TYPES[c["type"]])
    ids, p = _route(state)
    if op == "route":
        return ids.int(), p.float()
    x, M, E, I, K = state["x"].float(), c["M"], c["E"], c["I"], c["K"]
    if M * c["top_k"] <= E:
        # the chosen experts' weights alone, once for each slot
        slots = ids.flatten()
        gate, up, down = (_decode(state[n][0][slots], state[n][1][slots]) for n in ("gate", "up", "down"))
        xs = x.repeat_interleave(c["top_k"], 0)[:, None]
        g, u = (gate * xs).sum(-1), (up * xs).sum(-1)
        h = g / (1 + torch.exp(-g)) * u
        out = (down * h[:, None]).sum(-1)
        return (out.reshape(M, -1, K) * p.float()[..., None]).sum(1), ids.int(), p.float()
    # more slots than experts: every expert for every token, those not chosen with the weight zero
    gate, up, down = (_decode(*state[n]) for n in ("gate", "up", "down"))
    g, u = x @ gate.reshape(-1, K).T, x @ up.reshape(-1, K).T
    h = (g / (1 + torch.exp(-g)) * u).reshape(M, E, I)
    share = torch.zeros(M, E, device=x.device).scatter_(1, ids, p.float())
    y = (h * share[..., None]).reshape(M, -1) @ down.permute(0, 2, 1).reshape(-1, K)
    return y, ids.int(), p.float()


def work(case):
    op, K = case["op"], case["K"]
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["type"]]
    packed = 17 / 32   # bytes of a microscaled value: half a byte and its share of the scale
    if op == "quantise":
        # values read, planes written, planes read, 16-bit values written
        n = case["R"] * K
        return {"bytes": n * (size + 2 * packed + 2), "flops": 4 * n}
    if op == "gemv":
        M, N = case["M"], case["N"]
        return {"bytes": N * K * packed + M * K * size + M * N * 4, "flops": 2 * M * N * K}
    if op == "gemm":
        M, N = case["M"], case["N"]
        return {"bytes": (M + N) * K * packed + M * N * size, "flops": 2 * M * N * K}
    M, E, top_k = case["M"], case["E"], case["top_k"]
    b, f = (M + E) * K * size + M * top_k * 8, 2 * M * E * K
    if op == "moe":
        # experts that are read: those expected to be chosen by at least one of M tokens
        experts = E * (1 - (1 - top_k / E) ** M)
        b += experts * 3 * K * case["I"] * packed + M * K * 4
        f += 6 * M * top_k * K * case["I"]
    return {"bytes": b, "flops": f}


def _exact_values(codes, scales):
    """Values of the two planes in 64 bits, from the fields: sign, exponent, mantissa bit."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign = torch.where(c >= 8, -1.0, 1.0).double()
    c = c % 8
    e, m = torch.floor(c / 2), c % 2
    v = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    return sign * v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case["K"]
    if op == "quantise":
        x = s["x"].double().reshape(case["R"], -1, 32)
        amax = x.abs().amax(-1, keepdim=True)
        scale = torch.exp2((torch.floor(torch.log2(torch.where(amax > 0, amax, 2.0 ** -200))) - 2).clamp(-127, 127))
        a = x / scale
        # codes lie half a unit apart below 2, one up to 4, two above; round() goes to the even multiple
        step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
        return (torch.round(a / step) * step).clamp(-6, 6).mul(scale).reshape(case["R"], K)
    if op == "gemv":
        return s["x"].double() @ _exact_values(*s["w"]).T
    if op == "gemm":
        return _exact_values(*s["a"]) @ _exact_values(*s["w"]).T
    M, E, k = case["M"], case["E"], case["top_k"]
    x = s["x"].double()
    logits = (x[:, None, :] * s["router"].double()[None]).sum(-1) if M * E * K < 1 << 28 else x @ s["router"].double().T
    p = torch.softmax(logits, -1)
    # the number of experts ahead of each one: larger, or equal with a lower index
    at = torch.arange(E, device=x.device)
    ahead = (logits[:, None, :] > logits[:, :, None]) | ((logits[:, None, :] == logits[:, :, None]) & (at[None, None, :] < at[None, :, None]))
    rank = ahead.sum(-1)
    ids = torch.argsort(rank, -1)[:, :k]
    w = torch.gather(p, 1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    if op == "route":
        return ids.int(), w
    y = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        gate, up, down = (_exact_values(s[n][0][e], s[n][1][e]) for n in ("gate", "up", "down"))
        g = x[token] @ gate.T
        h = g * torch.sigmoid(g) * (x[token] @ up.T)
        y.index_add_(0, token, (h @ down.T) * w[token, slot][:, None])
    return y, ids.int(), w
