"""Cases that measure rotary positions, the paged key-value cache and the attention that reads it.

Four operators, each computed in two ways on the same inputs: through the
framework's calls where `own` is true, and otherwise in elementary torch
operations, in 32 bits (angles, rotations and the quantisation's divisions in
64: far positions and values next to a border).

  rope     kq_rope: rotary positions on the heads of a batch of tokens
  append   kq_kv_append, kq_kv_read: q and k of a fused q|k|v product rotated, k
           and v into the pages of a cache, and the rows just written read back
           as the values that the cache holds
  decode   kq_attn_decode: a few new tokens per sequence over the paged cache
  prompt   kq_attn_prompt: many new tokens per sequence, packed

The cache: pages of 32 positions, and in a page one region per key-value head,
laid out in pieces of 8 elements. With p the position in its page,
r = 4 (p / 8) + p % 4 and t = (p / 4) % 2:
  16-bit K   element (p, d) at (d / 32 * 2 + t) * 512 + (d % 32 / 8 * 16 + r) * 8 + d % 8
  16-bit V   element (p, d) at d / 16 * 512 + (p / 8 * 16 + d % 16) * 8 + p % 8
  Q8_0 K     byte (p, d) at d / 32 * 1024 + (d % 32 / 8 * 16 + r) * 16 + t * 8 + d % 8
  Q8_0 V     byte (p, d) at d / 32 * 1024 + (p / 8 * 16 + d % 16) * 16 + d % 32 / 16 * 8 + p % 8
  Q8_0       then the fp16 scales of 32 channels each, (p, b) at b * 32 + p
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAGE = 32


def listed():
    return [
        # q and k heads of a verify pass of 16 rows (32 + 8 heads of 128), straight from a product's fp32 rows.
        {"name": "rope_16x40x128_f32", "op": "rope", "tokens": 16, "heads": 40, "dim": 128, "rot": 128, "pairs": "half",
         "scaling": "none", "far": 4000, "type": "f32", "out": "f16"},
        # A prompt's queries with half of each head rotated, interleaved pairs, a context stretched fourfold.
        {"name": "rope_6001x32x128_bf16", "op": "rope", "tokens": 6001, "heads": 32, "dim": 128, "rot": 64,
         "pairs": "interleaved", "scaling": "yarn", "far": 131072, "type": "bf16", "out": "bf16"},
        # One layer of a verify pass: 16 rows of q|k|v (6144 wide) into an 8-bit cache.
        {"name": "append_16_q8_0", "op": "append", "seqs": 1, "queries": 16, "length": 5000, "heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "pairs": "half", "scaling": "none", "type": "f32", "cache": "q8_0", "out": "f16"},
        # One layer of seven packed prompts of different lengths.
        {"name": "append_7x700_bf16", "op": "append", "seqs": 7, "queries": 1100, "length": 1100, "heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "pairs": "half", "scaling": "linear", "type": "bf16", "cache": "bf16", "out": "bf16"},
        # One user's next token in a short chat: the call whose launch counts.
        {"name": "decode_1x1000_f16", "op": "decode", "seqs": 1, "queries": 1, "length": 1000, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0, "tree": False, "type": "f16", "cache": "f16"},
        # One user at the end of a stretched context of 131072.
        {"name": "decode_1x131071_bf16", "op": "decode", "seqs": 1, "queries": 1, "length": 131071, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "tree": False, "type": "bf16", "cache": "bf16"},
        # 48 requests of different lengths sharing a pass, 8-bit cache.
        {"name": "decode_48x8000_q8_0", "op": "decode", "seqs": 48, "queries": 1, "length": 8000, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0, "tree": False, "type": "f16", "cache": "q8_0"},
        # Three requests of 16 guessed tokens each, in trees.
        {"name": "decode_3x16_tree_f16", "op": "decode", "seqs": 3, "queries": 16, "length": 6000, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0, "tree": True, "type": "f16", "cache": "f16"},
        # Five short questions of different lengths in one pass.
        {"name": "prompt_5x150_f16", "op": "prompt", "seqs": 5, "queries": 150, "length": 150, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0, "type": "f16", "cache": "f16"},
        # A whole prompt of one user, one token short of a round size.
        {"name": "prompt_1x8191_bf16", "op": "prompt", "seqs": 1, "queries": 8191, "length": 8191, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "type": "bf16", "cache": "bf16"},
        # Twelve packed prompts through a layer with a sliding window, 8-bit cache, heads of 64.
        {"name": "prompt_12x2500_q8_0", "op": "prompt", "seqs": 12, "queries": 2500, "length": 2500, "heads": 16,
         "kv_heads": 4, "dim": 64, "window": 1000, "type": "f16", "cache": "q8_0"},
        # The last 500 tokens of a prompt read in chunks, 32 thousand before them in the cache.
        {"name": "prompt_1x500_behind_32000_bf16", "op": "prompt", "seqs": 1, "queries": 500, "length": 32500, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "type": "bf16", "cache": "bf16"},
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "prompt", "prompt"])
    dim = 32 * rng.choice([1, 2, 2, 3, 4, 4, 4, 5, 6, 7, 8])
    kind = rng.choice(["f16", "bf16"])
    turn = {"rot": rng.choice([dim, dim, 2 * rng.randint(1, dim // 2)]), "pairs": rng.choice(["half", "interleaved"]),
            "scaling": rng.choice(["none", "linear", "ntk", "yarn"])}
    if op == "rope":
        return {"op": op, "tokens": log_int(rng, 1, 6001), "heads": rng.randint(1, 40), "dim": dim, **turn,
                "far": log_int(rng, 1, 131072), "type": rng.choice(["f32", kind]), "out": rng.choice(["f32", "f16", "bf16"])}
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    shape = {"heads": kv_heads * rng.choice([1, 2, 3, 4, 5, 8]), "kv_heads": kv_heads, "dim": dim}
    cache = rng.choice([kind, kind, "q8_0"])
    if op == "append":
        seqs = log_int(rng, 1, 48)
        queries = log_int(rng, 1, max(1, 5000 // seqs))
        return {"op": op, "seqs": seqs, "queries": queries, "length": queries + rng.choice([0, log_int(rng, 1, 8000)]), **shape,
                **turn, "type": rng.choice(["f32", kind]), "cache": cache, "out": kind}
    window = rng.choice([0, 0, log_int(rng, 1, 4000)])
    if op == "decode":
        seqs = log_int(rng, 1, 64)
        queries = rng.choice([1, 1, rng.randint(1, 64 // seqs)])
        # the cached elements of all requests stay below those of the largest listed case
        most = min(131072, 48 * 8000 * 8 * 128 // (seqs * kv_heads * dim))
        return {"op": op, "seqs": seqs, "queries": queries, "length": log_int(rng, max(1, queries), most), **shape,
                "window": window, "tree": rng.random() < 0.3, "type": kind, "cache": cache}
    # scores of all requests stay below those of the largest listed case
    seqs = log_int(rng, 1, 24)
    queries = log_int(rng, 2, int(math.sqrt(8191 * 8191 * 32 * 128 / (seqs * shape["heads"] * dim * 2))))
    queries = min(queries, 8191)
    behind = rng.choice([0, 0, log_int(rng, 1, max(1, min(32000, 8191 * 8191 * 32 // (2 * seqs * queries * shape["heads"]))))])
    return {"op": op, "seqs": seqs, "queries": queries, "length": queries + behind, **shape, "window": window, "type": kind,
            "cache": cache}


def batch_of(case):
    """(new tokens, length) of each sequence: the first as the case says, the others shorter by parts that depend on the case alone."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["queries"], case["length"]))
    others, behind = range(case["seqs"] - 1), case["length"] - case["queries"]
    # verify passes give every request its rows; prompts differ in length
    new = [case["queries"]] + [case["queries"] if case["op"] == "decode" else rng.randint(1, case["queries"]) for _ in others]
    return new, [case["length"]] + [n + rng.randint(behind // 8, behind) for n in new[1:]]


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "q8_0": 34 / 32}
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": n * (size[case["type"]] + size[case["out"]]) + 4 * case["tokens"], "flops": 3 * n}
    new, lens = batch_of(case)
    T, H, Hk, D, held = sum(new), case["heads"], case["kv_heads"], case["dim"], size[case["cache"]]
    if case["op"] == "append":
        back = 4 if case["cache"] == "q8_0" else 2
        return {"bytes": T * D * ((H + 2 * Hk) * size[case["type"]] + H * size[case["out"]] + 2 * Hk * (2 * held + back)),
                "flops": 3 * T * (H + Hk) * case["rot"]}

    def pairs_of(n, length):
        """Visible (query, key) pairs: `few` queries see fewer keys than the window, the others a window full."""
        w = case["window"] or length
        first = length - n + 1
        few = max(0, min(n, w - first))
        return few * first + few * (few - 1) // 2 + (n - few) * w

    pairs = sum(map(pairs_of, new, lens))
    keys = sum(min(length, (case["window"] or length) + n - 1) for n, length in zip(new, lens))
    return {"bytes": 2 * keys * Hk * D * held + 2 * T * H * D * size[case["type"]], "flops": 4 * pairs * H * D}


# ---- inputs

def freqs_of(case):
    """(radians per position of each pair, factor on cos and sin), host values."""
    rot, base, factor, before = case["rot"], 1e6, 4.0, 32768
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "ntk":
        stretched = base * factor ** (rot / (rot - 2)) if rot > 2 else base
        return [stretched ** (-2 * i / rot) for i in range(rot // 2)], 1.0
    if case["scaling"] == "yarn":
        turns = [before * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / (32.0 - 1.0))) for t in turns]
        return [x * k + x / factor * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1
    return f, 1.0


def quantized(x):
    """Codes and scales (fp16) of blocks of 32 along the last axis, Q8_0; x: fp32."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    d = (b.abs().amax(-1).double() / 127).float().half()
    f = d.double()[..., None]
    ratio = (b.double() / torch.where(f == 0, 1.0, f)).float().double()
    codes = torch.where(f == 0, 0.0, (ratio.abs() + 0.5).floor() * ratio.sign()).clamp(-127, 127)
    return codes.to(torch.int8).reshape(x.shape), d


def into_pages(k, kind, is_v):
    """Rows [pages][positions][heads][dim] as the pages' bytes [pages][heads][...]."""
    P, _, H, D = k.shape

    def order(e):
        e = e.reshape(P, 4, 2, 4, H, D // 32, 4, 8) if not is_v else e
        if kind == "q8_0":
            if is_v:   # p / 8, p % 8, head, block, half, d % 16 -> head, block, p / 8, d % 16, half, p % 8
                return e.reshape(P, 4, 8, H, D // 32, 2, 16).permute(0, 3, 4, 1, 6, 5, 2)
            return e.permute(0, 4, 5, 6, 1, 3, 2, 7)   # head, block, d piece, p / 8, p % 4, t, d % 8
        if is_v:
            return e.reshape(P, 4, 8, H, D // 16, 16).permute(0, 3, 4, 1, 5, 2)
        return e.permute(0, 4, 5, 2, 6, 1, 3, 7)

    if kind == "q8_0":
        codes, d = quantized(k.float())
        codes = order(codes).reshape(P, H, 32 * D).contiguous().view(torch.uint8)
        scales = d.permute(0, 2, 3, 1).reshape(P, H, D).contiguous().view(torch.uint8)
        return torch.cat([codes, scales], -1).contiguous()
    return order(k.to(TYPES[kind])).reshape(P, H, 32 * D).contiguous().view(torch.uint8)


def prepare(case, seed):
    def tree_of(n):
        """Bit masks of n guessed tokens: each sees its ancestors and itself."""
        rng, masks = random.Random(seed), []
        for i in range(n):
            masks.append((masks[rng.randint(0, i - 1)] if i else 0) | 1 << i)
        return [m - (1 << 64) if m >> 63 else m for m in masks]

    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] in ("rope", "append"):
        freqs, s["mscale"] = freqs_of(case)
        s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    if case["op"] == "rope":
        T = case["tokens"]
        s["x"] = normal(T, case["heads"] * case["dim"]).to(TYPES[case["type"]])
        start = random.Random(seed).randint(0, case["far"])
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        s["y"] = torch.empty(T, case["heads"] * case["dim"], dtype=TYPES[case["out"]], device="cuda")
        return s
    new, lens = batch_of(case)
    S, T, H, Hk, D = case["seqs"], sum(new), case["heads"], case["kv_heads"], case["dim"]
    width = -(-max(lens) // PAGE)
    counts = [-(-n // PAGE) for n in lens]
    pages = sum(counts)
    # a sequence's pages lie anywhere in the cache; table entries past its length name any page
    where = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(counts[:i]) for i in range(S)], device="cuda")
    s["table"] = where[(first[:, None] + torch.arange(width, device="cuda")).clamp(max=pages - 1)].contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
    s.update(pages=pages, width=width, tokens=T, most_new=max(new))
    if case["op"] == "append":
        s["qkv"] = normal(T, (H + 2 * Hk) * D).to(TYPES[case["type"]])
        page_bytes = Hk * D * (34 if case["cache"] == "q8_0" else 64)
        s["k"] = torch.zeros(pages, page_bytes, dtype=torch.uint8, device="cuda")
        s["v"] = torch.zeros(pages, page_bytes, dtype=torch.uint8, device="cuda")
        back = torch.float32 if case["cache"] == "q8_0" else TYPES[case["cache"]]
        s["k_back"], s["v_back"] = (torch.empty(T, Hk * D, dtype=back, device="cuda") for _ in range(2))
        s["out"] = torch.empty(T, H * D, dtype=TYPES[case["out"]], device="cuda")
        return s
    s["k"], s["v"] = (torch.cat([into_pages(normal(min(2048, pages - i), PAGE, Hk, D), case["cache"], is_v)
                                 for i in range(0, pages, 2048)]) for is_v in (False, True))
    # queries lean towards a few keys, as trained heads do: scores with a spread of about 2
    s["q"] = (normal(T, H * D) * 2).to(TYPES[case["type"]])
    s["out"] = torch.empty(T, H * D, dtype=TYPES[case["type"]], device="cuda")
    s["scale"] = D ** -0.5
    s["tree"] = None
    if case.get("tree"):
        s["tree"] = torch.tensor([m for n in new for m in tree_of(n)], dtype=torch.int64, device="cuda")
    return s


# ---- the framework's calls

def run_own(s):
    import block_quantized_gemv_kq_amd as kq
    case = s["case"]
    H, D = case["heads"], case["dim"]
    pairs = kq.KQ_ROPE_HALF if case.get("pairs") == "half" else kq.KQ_ROPE_INTERLEAVED
    if case["op"] == "rope":
        rope = kq.kq_rope_spec(s["freqs"], case["rot"], pairs, s["mscale"], s["positions"])
        kq.kq_rope(rope, case["type"], s["x"], H * D, case["out"], s["y"], H * D, case["tokens"], H, D)
        return s["y"]
    Hk, T = case["kv_heads"], s["tokens"]
    cache = kq.kq_kv_cache(case["cache"], s["k"], s["v"], s["pages"], Hk, D)
    batch = kq.kq_kv_batch(s["table"], s["width"], s["q_start"], s["lens"], case["seqs"], T)
    if case["op"] == "append":
        rope = kq.kq_rope_spec(s["freqs"], case["rot"], pairs, s["mscale"])
        row = (H + 2 * Hk) * D
        q, k, v = s["qkv"], s["qkv"][:, H * D:], s["qkv"][:, (H + Hk) * D:]
        kq.kq_kv_append(cache, batch, rope, case["type"], k, row, v, row, q, row, case["out"], s["out"], H * D, H)
        kq.kq_kv_read(cache, batch, "f32" if case["cache"] == "q8_0" else case["cache"], s["k_back"], Hk * D, s["v_back"],
                      Hk * D)
        return s["out"], s["k_back"], s["v_back"]
    if "workspace" not in s:   # the first call's, kept
        need = (kq.kq_attn_decode_workspace_bytes if case["op"] == "decode" else kq.kq_attn_prompt_workspace_bytes)(
            cache, batch, H)
        s["workspace"], s["workspace_bytes"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), need
    if case["op"] == "decode":
        kq.kq_attn_decode(case["type"], s["q"], H * D, cache, batch, s["out"], H * D, H, s["scale"], case["window"], s["tree"],
                          s["workspace"], s["workspace_bytes"])
    else:
        kq.kq_attn_prompt(case["type"], s["q"], H * D, cache, batch, s["out"], H * D, H, s["scale"], case["window"],
                          s["workspace"], s["workspace_bytes"])
    return s["out"]


# ---- the plain forms

def turned(x, positions, s):
    """x [tokens][heads][dim] (64 bits) rotated."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    angle = positions.double()[:, None] * s["freqs"]
    cos, sin = (angle.cos() * s["mscale"])[:, None], (angle.sin() * s["mscale"])[:, None]
    part = x[..., :rot]
    if s["case"]["pairs"] == "half":
        a, b = part[..., :half], part[..., half:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([part, x[..., rot:]], -1)


def whereabouts(s):
    """(sequence, index among its new tokens, position) of each token."""
    token = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), token, right=True)
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    index = token - s["q_start"].long()[seq]
    return seq, index, s["lens"].long()[seq] - new[seq] + index


def dense(pages, s, is_v):
    """The cache's values [sequences][kv heads][positions][dim] in 32 bits, by the page table."""
    case, (S, W) = s["case"], s["table"].shape
    H, D = case["kv_heads"], case["dim"]
    held = pages.view(s["pages"], H, -1)[s["table"].long()]
    if case["cache"] == "q8_0":
        codes = held[..., :32 * D].contiguous().view(torch.int8)
        scales = held[..., 32 * D:].contiguous().view(torch.float16).view(S, W, H, D // 32, 32).float()
        if is_v:
            e = codes.view(S, W, H, D // 32, 4, 16, 2, 8).permute(0, 2, 1, 4, 7, 3, 6, 5)
        else:
            e = codes.view(S, W, H, D // 32, 4, 4, 4, 2, 8).permute(0, 2, 1, 5, 7, 6, 3, 4, 8)
        e = e.reshape(S, H, W * 32, D // 32, 32).float()
        return (e * scales.permute(0, 2, 1, 4, 3).reshape(S, H, W * 32, D // 32, 1)).reshape(S, H, W * 32, D)
    e = held.view(TYPES[case["cache"]])
    if is_v:
        e = e.view(S, W, H, D // 16, 4, 16, 8).permute(0, 2, 1, 4, 6, 3, 5)
    else:
        e = e.view(S, W, H, D // 32, 2, 4, 4, 4, 8).permute(0, 2, 1, 6, 4, 7, 3, 5, 8)
    return e.reshape(S, H, W * 32, D).float()


def attention(s):
    case = s["case"]
    S, n, H, Hk, D = case["seqs"], s["most_new"], case["heads"], case["kv_heads"], case["dim"]
    k, v = dense(s["k"], s, False), dense(s["v"], s, True)
    token = (s["q_start"][:-1].long()[:, None] + torch.arange(n, device="cuda")).clamp(max=s["tokens"] - 1)
    q = s["q"].view(-1, Hk, H // Hk, D)[token].float().permute(0, 2, 3, 1, 4).reshape(S, Hk, -1, D)
    scores = (torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]).view(S, Hk, H // Hk, n, -1)
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    at = (s["lens"].long() - new)[:, None] + torch.arange(n, device="cuda")
    key = torch.arange(scores.shape[-1], device="cuda")
    seen = key <= at[..., None]
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    if s["tree"] is not None:
        among = key - (s["lens"].long() - new)[:, None]          # index among the new tokens, negative before them
        bit = (s["tree"][token][..., None] >> among.clamp(0, 63)[:, None]) & 1
        seen &= (among < 0)[:, None] | (bit == 1)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    most = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(S, Hk, -1, scores.shape[-1]), v).view(S, Hk, H // Hk, n, D)
    out = torch.where(total > 0, out / total, 0.0)
    seq, index, _ = whereabouts(s)
    return out.permute(0, 3, 1, 2, 4)[seq, index].reshape(s["tokens"], H * D).to(TYPES[case["type"]])


def run(s):
    if own:
        return run_own(s)
    case = s["case"]
    H, D = case["heads"], case["dim"]
    if case["op"] == "rope":
        x = s["x"].view(-1, H, D).double()
        return turned(x, s["positions"], s).to(TYPES[case["out"]]).view(-1, H * D)
    if case["op"] != "append":
        return attention(s)
    Hk, position = case["kv_heads"], whereabouts(s)[2]
    q, k, v = (x.reshape(s["tokens"], -1, D) for x in s["qkv"].split([H * D, Hk * D, Hk * D], -1))
    q = turned(q.double(), position, s).to(TYPES[case["out"]])
    k = turned(k.double(), position, s)
    if case["cache"] == "q8_0":
        (kc, kd), (vc, vd) = quantized(k.float()), quantized(v.float())
        k, v = (c.float() * d.float().repeat_interleave(32, -1) for c, d in ((kc, kd), (vc, vd)))
    else:
        k, v = k.to(TYPES[case["cache"]]), v.to(TYPES[case["cache"]])
    return q.reshape(-1, H * D), k.reshape(-1, Hk * D), v.reshape(-1, Hk * D)


# ---- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    H, D = case["heads"], case["dim"]

    def rotate(x, position):
        """One token's heads [heads][dim] by complex multiplication."""
        rot, w = case["rot"], torch.polar(torch.full_like(s["freqs"], s["mscale"]), s["freqs"] * float(position))
        even, odd = (slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[:, even].contiguous(), x[:, odd].contiguous()) * w
        y = x.clone()
        y[:, even], y[:, odd] = z.real, z.imag
        return y

    if case["op"] == "rope":
        x = s["x"].double().view(-1, H, D)
        return torch.stack([rotate(row, p) for row, p in zip(x, s["positions"].tolist())]).view(-1, H * D)
    Hk, T = case["kv_heads"], s["tokens"]
    new, lens = batch_of(case)
    if case["op"] == "append":
        positions = [length - n + i for n, length in zip(new, lens) for i in range(n)]
        rows = s["qkv"].double().view(T, H + 2 * Hk, D)
        q = torch.stack([rotate(r[:H], p) for r, p in zip(rows, positions)])
        if case["cache"] == "q8_0":
            return q.view(T, -1), None, None   # what 8 bits hold is compared with the plain form's
        k = torch.stack([rotate(r[H:H + Hk], p) for r, p in zip(rows, positions)])
        return q.view(T, -1), k.view(T, -1), rows[:, H + Hk:].reshape(T, -1)
    # the place of each (position, channel) in a page's region, by the formulas above
    p, d = torch.arange(32, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    r, t = 4 * (p // 8) + p % 4, p // 4 % 2
    if case["cache"] == "q8_0":
        k_at = d // 32 * 1024 + (d % 32 // 8 * 16 + r) * 16 + t * 8 + d % 8
        v_at = d // 32 * 1024 + (p // 8 * 16 + d % 16) * 16 + d % 32 // 16 * 8 + p % 8
    else:
        k_at = (d // 32 * 2 + t) * 512 + (d % 32 // 8 * 16 + r) * 8 + d % 8
        v_at = d // 16 * 512 + (p // 8 * 16 + d % 16) * 8 + p % 8
    out = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
    begin = 0
    for i, (n, length) in enumerate(zip(new, lens)):
        pages = s["table"][i, :-(-length // 32)].long()
        at = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        seen = (key <= at) & ((key > at - case["window"]) if case["window"] else True)
        if s["tree"] is not None:
            masks = [m & (1 << 64) - 1 for m in s["tree"][begin:begin + n].tolist()]
            seen[:, length - n:] &= torch.tensor([[m >> j & 1 == 1 for j in range(n)] for m in masks], device="cuda")
        for h in range(Hk):
            kv = []
            for held, where in ((s["k"], k_at), (s["v"], v_at)):
                region = held.view(s["pages"], Hk, -1)[pages, h]
                if case["cache"] == "q8_0":
                    scales = region[:, 32 * D:].contiguous().view(torch.float16).double()
                    e = region[:, where].view(torch.int8).double() * scales[:, d // 32 * 32 + p]
                else:
                    e = region.view(TYPES[case["cache"]])[:, where].double()
                kv.append(e.reshape(-1, D)[:length])
            for j in range(h * (H // Hk), (h + 1) * (H // Hk)):
                q = s["q"][begin:begin + n, j * D:(j + 1) * D].double()
                weights = torch.softmax(torch.where(seen, q @ kv[0].T * s["scale"], -math.inf), -1)
                out[begin:begin + n, j] = torch.where(seen, weights, 0.0) @ kv[1]
        begin += n
    return out.view(T, H * D)
