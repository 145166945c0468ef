"""Operators over a paged cache of E4M3 codes with a scale for each block of tokens and head: cases, plain forms and work.

A pool holds codes [num_pages, num_kv_heads, page_size, head_dim]; `block` consecutive rows of a page and kv head share
one float32 scale, [num_pages, num_kv_heads, page_size / block]; an element is its code's value times its block's scale.

- rotate: q and k heads normalised (root mean square, a weight per element) and rotated in one pass;
- append: new tokens (one, a draft, a prompt per request) normalised, rotated and written into their pages: quantised
  into such pools (the scale of a block follows its largest element as rows arrive), or as they are;
- read: tokens of such a cache read back as f16, bf16 or f32 rows;
- decode: one query token per request over such a cache;
- tree: a request's last tokens at once (a chain, a piece of a prompt, or a tree given by a bit mask).

`run` computes a case either in plain torch operations (own = False) or with the framework's calls (own = True), on the
same state.
"""
import math
import statistics

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
#: One scratch buffer of a serving program, for every call on its stream.
WORKSPACE = 192 << 20
EPS = 1e-6
#: Smallest scale of a block; the largest code; what still rounds to it.
LEAST, TOP, EDGE = 2.0 ** -126, 448.0, 464.0


# ---------------------------------------------------------------- cases

def listed():
    base = {"theta": 500000.0, "layout": "half", "scaling": "none"}
    llama = {"hq": 32, "hk": 8, "d": 128, "page": 16, "block": 16}
    seventy = {"hq": 64, "hk": 8, "d": 128, "page": 32, "block": 32}
    return [
        # one decoded token far into a long context
        {"name": "rotate_one_token", "op": "rotate", "tokens": 1, "hq": 32, "hk": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "far": 131071, **base},
        # a prompt of odd length, pairs side by side, half of each head rotated, stretched context
        {"name": "rotate_prompt_f16", "op": "rotate", "tokens": 8191, "hq": 56, "hk": 8, "d": 128, "rot": 64, "dtype": "f16",
         "far": 8191, **base, "layout": "pairs", "scaling": "yarn"},
        # the batched decode step: one token for each of 32 requests, most of them into a block that holds rows already
        {"name": "append_b32_bf16", "op": "append", "batch": 32, "new_lo": 1, "new_hi": 1, "kv_lo": 512, "kv_hi": 4096,
         "spread": "uniform", **llama, "rot": 128, "dtype": "bf16", "norm": True, "positions": "given", **base,
         "scaling": "banded"},
        # ragged prompts and drafts together
        {"name": "append_prompts_f16", "op": "append", "batch": 24, "new_lo": 1, "new_hi": 4095, "kv_lo": 1, "kv_hi": 4095,
         "spread": "log", **seventy, "rot": 128, "dtype": "f16", "norm": True, "positions": "index", **base,
         "layout": "pairs"},
        # the same traffic into a pool of the rows' own type
        {"name": "append_prompts_plain_bf16", "op": "append", "batch": 24, "new_lo": 1, "new_hi": 4095, "kv_lo": 1,
         "kv_hi": 4095, "spread": "log", **llama, "block": 0, "rot": 128, "dtype": "bf16", "norm": True,
         "positions": "index", **base},
        # one short request, a scale for each token
        {"name": "read_tiny_f32", "op": "read", "batch": 1, "kv_lo": 100, "kv_hi": 100, "spread": "uniform", "hq": 8, "hk": 2,
         "d": 64, "page": 16, "block": 1, "dtype": "f32", "piece": "all"},
        # what a prompt's cache holds, for attention in 16 bits or for a copy elsewhere
        {"name": "read_b16_bf16", "op": "read", "batch": 16, "kv_lo": 512, "kv_hi": 16384, "spread": "log", **llama,
         "dtype": "bf16", "piece": "part"},
        # the smallest call: one request of 100 tokens
        {"name": "decode_tiny_f16", "op": "decode", "batch": 1, "kv_lo": 100, "kv_hi": 100, "spread": "uniform", "hq": 8,
         "hk": 2, "d": 64, "page": 16, "block": 16, "dtype": "f16", "empty": False},
        # the batched decode step
        {"name": "decode_b32_bf16", "op": "decode", "batch": 32, "kv_lo": 512, "kv_hi": 4096, "spread": "uniform", **llama,
         "dtype": "bf16", "empty": False},
        # four long contexts
        {"name": "decode_long_b4_f16", "op": "decode", "batch": 4, "kv_lo": 131071, "kv_hi": 131071, "spread": "uniform",
         **llama, "dtype": "f16", "empty": False},
        # trees of 1 to 32 nodes, a large ragged batch, groups of 8 heads
        {"name": "tree_b64_bf16", "op": "tree", "batch": 64, "new_lo": 1, "new_hi": 32, "kv_lo": 32, "kv_hi": 8192,
         "spread": "lognormal", **seventy, "dtype": "bf16", "mask": "tree"},
        # pieces of four prompts over what is cached of them
        {"name": "tree_chunk_bf16", "op": "tree", "batch": 4, "new_lo": 1021, "new_hi": 1021, "kv_lo": 7000, "kv_hi": 8191,
         "spread": "uniform", **llama, "dtype": "bf16", "mask": "chain"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "append", "read", "decode", "decode", "decode", "tree", "tree"])
    hq, hk, d, page = rng.choice([(32, 8, 128, 16), (64, 8, 128, 32), (16, 16, 256, 16), (8, 2, 64, 16), (28, 4, 128, 16),
                                  (32, 8, 128, 64), (12, 4, 64, 8), (32, 2, 128, 16)])
    block = rng.choice([b for b in (page, page, page, 16, 4, 1) if page % b == 0])
    shape = {"hq": hq, "hk": hk, "d": d, "page": page, "block": block}
    dtype = rng.choice(["f16", "bf16", "bf16"])
    rope = {"rot": rng.choice([d, d, d // 2]), "theta": rng.choice([10000.0, 500000.0]),
            "layout": rng.choice(["half", "pairs"]), "scaling": rng.choice(["none", "linear", "banded", "yarn"])}
    if op == "rotate":
        tokens = _log(rng, 1, 8191)
        return {"op": op, "tokens": tokens, "hq": hq, "hk": hk, "d": d, "dtype": rng.choice([dtype, dtype, "f32"]),
                "far": max(tokens, _log(rng, 64, 131071)), **rope}
    batch = _log(rng, 1, 64)
    if op == "append":
        hi = _log(rng, 1, max(1, 16384 // batch))
        plain = rng.random() < 0.25
        lo = hi // 4 if batch >= 8 else max(1, hi // 4)  # some requests of a batch bring nothing
        return {"op": op, "batch": batch, "new_lo": lo, "new_hi": hi, "kv_lo": hi,
                "kv_hi": hi + _log(rng, 1, 2048), "spread": "uniform", **shape, "block": 0 if plain else block,
                "dtype": rng.choice([dtype, "f32"]) if plain else dtype, "norm": plain or rng.random() < 0.6,
                "positions": rng.choice(["given", "index"]), **rope}
    if op == "read":
        hi = _log(rng, 64, 131072 // batch)
        return {"op": op, "batch": batch, "kv_lo": max(1, hi // 8), "kv_hi": hi, "spread": "log", **shape,
                "dtype": rng.choice([dtype, dtype, "f32"]), "piece": rng.choice(["all", "part"])}
    if op == "decode":
        hi = _log(rng, 16, min(131072, 524288 // batch))
        return {"op": op, "batch": batch, "kv_lo": max(1, hi // 8), "kv_hi": hi, "spread": rng.choice(["uniform", "log"]),
                **shape, "dtype": dtype, "empty": batch > 1 and rng.random() < 0.3}
    mask = rng.choice(["tree", "chain"])
    hi = _log(rng, 1, 64) if mask == "tree" else _log(rng, 1, 1024)
    tokens = min(131072 * 4 // batch, max(64, int(2.0e11 / (hi * hq * d * 4 * batch))))
    kv = hi + _log(rng, 16, min(131072, tokens))
    lo = hi // 3 if batch >= 8 else max(1, hi // 3)
    return {"op": op, "batch": batch, "new_lo": lo, "new_hi": hi, "kv_lo": hi + (kv - hi) // 4, "kv_hi": kv,
            "spread": rng.choice(["uniform", "log"]), **shape, "dtype": dtype, "mask": mask}


def _lengths(case):
    """(kv_len, new) of each request: spread over the case's range by low-discrepancy points, the same for every seed."""
    b = case["batch"]
    u = (np.arange(b) * 0.6180339887498949 + 0.5) % 1.0
    lo, hi = case["kv_lo"], case["kv_hi"]
    if case["spread"] == "uniform":
        kv = lo + u * (hi - lo)
    elif case["spread"] == "log":
        kv = np.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))
    else:
        z = np.array([statistics.NormalDist().inv_cdf(min(max(x, 1e-3), 1 - 1e-3)) for x in u])
        kv = np.clip(1024.0 * np.exp(z), lo, hi)
    kv = np.maximum(1, np.rint(kv)).astype(np.int64)
    if case.get("empty"):
        kv[b // 2] = 0
    w = (np.arange(b) * 0.7548776662466927 + 0.25) % 1.0
    if case["op"] == "decode":
        new = np.ones(b, np.int64)
    elif case["op"] == "read":
        new = np.maximum(1, np.rint(kv * (0.5 + 0.5 * w))).astype(np.int64) if case["piece"] == "part" else kv
    else:
        new = np.rint(case["new_lo"] + w * (case["new_hi"] - case["new_lo"])).astype(np.int64)
    return kv, (new if case["op"] == "decode" else np.minimum(new, kv))


def work(case):
    op = case["op"]
    e, heads = SIZE[case["dtype"]], case["hq"] + case["hk"]
    if op == "rotate":
        return {"bytes": 2 * case["tokens"] * heads * case["d"] * e + 4 * case["tokens"],
                "flops": case["tokens"] * heads * (4 * case["d"] + 3 * case["rot"])}
    kv, new = _lengths(case)
    pages = int(np.sum(-(-kv // case["page"])))
    table = 4 * (pages + 2 * case["batch"] + 1 + case["batch"] + 1)
    row, q, t, block = case["hk"] * case["d"], case["hq"] * case["d"], int(new.sum()), case["block"]

    def scales(tokens):  # of the blocks that hold them, K and V
        return 2 * 4 * case["hk"] * (-(-tokens // block)) if block else 0

    if op == "append":
        return {"bytes": t * (2 * q * e + 2 * row * (e + (1 if block else e))) + scales(t) + table,
                "flops": t * heads * (3 * case["rot"] + (4 * case["d"] if case["norm"] else 0))}
    if op == "read":
        return {"bytes": t * 2 * row * (1 + e) + scales(t) + table, "flops": 2 * t * row}
    if op == "decode":
        pairs = int(kv.sum())
    else:
        pairs = int(np.sum(new * (kv - new) + (new * (new + 1)) // 2))  # a tree sees fewer of its own nodes
    return {"bytes": 2 * int(kv.sum()) * row + scales(int(kv.sum())) + 2 * t * q * e + 4 * t * case["hq"] + table,
            "flops": 4 * case["d"] * case["hq"] * pairs}


# ---------------------------------------------------------------- inputs

def _inv_freq(case):
    """Radians per position of each pair (64 bits) and the factor on the rotated part, from the case's scaling."""
    rot, theta, factor, original = case["rot"], case["theta"], 8.0, 8192
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "banded":  # long wavelengths stretched, short ones kept, a ramp between
        turns = original * f / (2 * math.pi)
        s = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return (1 - s) * f / factor + s * f, 1.0
    if case["scaling"] == "yarn":  # the ramp over the pair's index, between 32 and 1 turns in the original context
        at = [rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        s = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return s * f / factor + (1 - s) * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def _tree(n, rng):
    """Parents of a drafted tree in breadth-first order: each node hangs from one of the few before it."""
    p = np.arange(n) - 1 - (rng.random(n) * np.minimum(6, np.arange(n) + 1)).astype(np.int64)
    return np.maximum(p, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": dict(case)}
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]

    def normal(shape, dtype):
        return torch.randn(shape, device="cuda", dtype=TYPES[dtype], generator=gen)

    def rand(shape):
        return torch.rand(shape, device="cuda", generator=gen)

    if "rot" in case:
        inv, factor = _inv_freq(case)
        # the framework's table: each pair's turns per position, in units of 2^-64 turn
        s["freqs"] = torch.from_numpy(np.ldexp(inv / (2 * math.pi), 64).astype(np.uint64).view(np.int64)).cuda()
        s["inv"], s["factor"] = torch.from_numpy(inv).cuda(), factor
        s["q_weight"], s["k_weight"] = (1 + 0.2 * normal((d,), case["dtype"]) for _ in range(2))
    if op == "rotate":
        t = case["tokens"]
        # one projection's output holds q, k and v of a token side by side
        qkv = normal((t, hq + 2 * hk, d), case["dtype"])
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        first = max(0, case["far"] - t + 1 - int(rng.integers(0, 32)))
        s["positions"] = _i32(first + np.arange(t))
        s["q_out"] = torch.empty(t, hq, d, dtype=TYPES[case["dtype"]], device="cuda")
        s["k_out"] = torch.empty(t, hk, d, dtype=TYPES[case["dtype"]], device="cuda")
        return s
    page, block = case["page"], case["block"]
    kv, new = _lengths(case)
    # a shuffled page table over a pool of a tenth more pages than are used
    n = -(-kv // page)
    used = int(n.sum())
    total = used + max(1, used // 10)
    s["indices"], s["indptr"] = _i32(rng.permutation(total)[:used]), _i32(np.concatenate([[0], np.cumsum(n)]))
    s["last"] = _i32(np.where(n > 0, kv - (n - 1) * page, 0))
    starts = np.concatenate([[0], np.cumsum(new)])
    s["new_indptr"] = _i32(starts)
    # on the host, a program knows its requests' lengths
    s["kv"], s["new"] = kv, new
    t = int(new.sum())
    if block:  # values of magnitude 1 / 2 to 2, by block
        for x in ("k", "v"):
            s[x] = (torch.randn(total, hk, page, d, device="cuda", dtype=torch.float16, generator=gen) * 64).clamp(
                -448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[x + "_scale"] = torch.exp2(2 * rand((total, hk, page // block)) - 7)
    else:
        s["k"], s["v"] = (normal((total, hk, page, d), case["dtype"]) for _ in range(2))
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    if op == "append":
        qkv = normal((t, hq + 2 * hk, d), case["dtype"])
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(t, hq, d, dtype=TYPES[case["dtype"]], device="cuda")
        s["positions"] = None
        if case["positions"] == "given":
            s["positions"] = _i32(np.concatenate([np.arange(m) + (l - m) for l, m in zip(kv, new)]) + 60000)
    elif op == "read":
        s["first"] = _i32(kv - new) if case["piece"] == "part" else None
        s["k_out"], s["v_out"] = (torch.empty(t, hk, d, dtype=TYPES[case["dtype"]], device="cuda") for _ in range(2))
    else:
        s["q"] = normal((t, hq, d), case["dtype"])
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(t, hq, device="cuda")
        s["mask"] = None
        if op == "tree" and case["mask"] == "tree":
            words = max(1, -(-int(new.max()) // 32))
            bits = np.zeros((t, words), np.uint32)
            for b, m in enumerate(new):
                for j, p in enumerate(_tree(int(m), rng)):
                    if p >= 0:
                        bits[starts[b] + j] = bits[starts[b] + p]
                    bits[starts[b] + j, j // 32] |= np.uint32(1 << (j % 32))
            s["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, weight, positions, s, wide=torch.float32):
    """Heads divided by the root of their mean square (weight given), then each pair turned."""
    c, x = s["case"], x.to(wide)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(wide)
    angle = positions.double()[:, None] * s["inv"]
    cos, sin = ((f * s["factor"]).to(wide)[:, None] for f in (angle.cos(), angle.sin()))
    rot = c["rot"]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if c["layout"] == "half" else (x[..., :rot:2], x[..., 1:rot:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rows(s, request, token):
    """(page, row) of a request's token."""
    page = s["case"]["page"]
    return s["indices"].long()[s["indptr"].long()[request] + token // page], token % page


def _ragged(s):
    """For each new token: its request, its index among the request's new tokens; the requests' lengths and new tokens."""
    start = s["new_indptr"].long()
    new = start[1:] - start[:-1]
    request = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new, output_size=int(s["new"].sum()))
    nth = torch.arange(request.numel(), device="cuda") - start[request]
    pages = (s["indptr"][1:] - s["indptr"][:-1]).long()
    kv = torch.where(pages > 0, (pages - 1) * s["case"]["page"] + s["last"].long(), 0)
    return request, nth, kv, new


def _code(x):
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, wide=torch.float32):
    return codes.view(torch.float8_e4m3fn).to(wide)


def _into_blocks(pool, scales, x, page, row, s, request, kv, new):
    """Rows x (64 bits) into their blocks: scales first, then rows that were there under a scale that grew, then x."""
    c = s["case"]
    block = c["block"]
    per = c["page"] // block
    ctx = kv - new
    flat = scales.permute(0, 2, 1).flatten(0, 1).double()  # [block, head]
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    at = page * per + row // block
    most = torch.zeros_like(flat).scatter_reduce_(0, at[:, None].expand_as(top), top, "amax")
    # a request's rows that share a block with its first new one
    n_old = torch.where(new > 0, ctx % block, 0)
    places = torch.arange(block, device="cuda")
    inside = places < n_old[:, None]
    old_page, old_row = _rows(s, torch.arange(c["batch"], device="cuda")[:, None],
                              torch.where(inside, (ctx - n_old)[:, None] + places, 0))
    old_page, old_row = old_page[inside], old_row[inside]
    old_at = old_page * per + old_row // block
    kept = torch.zeros(flat.shape[0], 1, dtype=torch.bool, device="cuda")
    kept[old_at] = True
    wanted = (most / TOP).clamp(min=LEAST).float().double()
    before = flat.clamp(min=LEAST)
    grown = before * torch.exp2(torch.log2(most / (EDGE * before)).ceil().clamp(min=0))
    touched = torch.zeros_like(kept)
    touched[at] = True
    after = torch.where(touched, torch.where(kept, grown, wanted), flat)
    ratio = (before / after)[old_at][..., None]
    pool[old_page, :, old_row] = _code(_value(pool[old_page, :, old_row], torch.float64) * ratio)
    pool[page, :, row] = _code(x / after[at][..., None])
    scales.copy_(after.unflatten(0, (-1, per)).permute(0, 2, 1))


def _plain_append(s):
    c = s["case"]
    request, nth, kv, new = _ragged(s)
    token = kv[request] - new[request] + nth
    at = token if s["positions"] is None else s["positions"]
    qw, kw = (s["q_weight"], s["k_weight"]) if c["norm"] else (None, None)
    s["q_out"].copy_(_rotate(s["q"], qw, at, s))
    page, row = _rows(s, request, token)
    if c["block"]:  # a code's rounding border is near many values
        _into_blocks(s["k"], s["k_scale"], _rotate(s["k_new"], kw, at, s, torch.float64), page, row, s, request, kv, new)
        _into_blocks(s["v"], s["v_scale"], s["v_new"].double(), page, row, s, request, kv, new)
    else:
        s["k"][page, :, row] = _rotate(s["k_new"], kw, at, s).to(s["k"].dtype)
        s["v"][page, :, row] = s["v_new"]


def _tokens_of(s, pool, scales, page, row):
    """[..., head, dim] values of the cache's tokens at (page, row)."""
    return _value(pool[page, :, row]) * scales[page, :, row // s["case"]["block"]][..., None]


def _plain_read(s):
    request, nth, _, _ = _ragged(s)
    token = nth if s["first"] is None else s["first"].long()[request] + nth
    page, row = _rows(s, request, token)
    s["k_out"].copy_(_tokens_of(s, s["k"], s["k_scale"], page, row))
    s["v_out"].copy_(_tokens_of(s, s["v"], s["v_scale"], page, row))


def _plain_attend(s):
    c = s["case"]
    request, nth, kv, new = _ragged(s)
    most, wide, group = int(s["kv"].max()), int(s["new"].max()), c["hq"] // c["hk"]
    token = torch.arange(most, device="cuda")
    inside = token < kv[:, None]
    page, row = _rows(s, torch.where(kv > 0, torch.arange(c["batch"], device="cuda"), int(s["kv"].argmax()))[:, None],
                      torch.where(inside, token, 0))
    k = _tokens_of(s, s["k"], s["k_scale"], page, row).permute(0, 2, 1, 3)  # [batch, head, token, dim]
    v = _tokens_of(s, s["v"], s["v_scale"], page, row).permute(0, 2, 1, 3)
    q = torch.zeros(c["batch"], wide, c["hq"], c["d"], device="cuda")
    q[request, nth] = s["q"].float()
    q = q.view(c["batch"], wide, c["hk"], group, c["d"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    node = token - (kv - new)[:, None]  # index among the new rows
    if s["mask"] is None:
        seen = node[:, None, :] <= torch.arange(wide, device="cuda")[:, None]
    else:
        bits = torch.zeros(c["batch"], wide, s["mask"].shape[1], dtype=torch.int32, device="cuda")
        bits[request, nth] = s["mask"]
        at = node.clamp(min=0, max=32 * s["mask"].shape[1] - 1)
        words = bits.gather(2, (at // 32)[:, None, :].expand(-1, wide, -1))
        seen = (node < 0)[:, None, :] | (((words >> (at % 32)[:, None, :].int()) & 1) != 0)
    seen = (seen & inside[:, None, :])[:, None, None]  # [batch, 1, 1, node, token]
    x = (q @ k.transpose(2, 3) * (1 / math.sqrt(c["d"]))).unflatten(2, (group, wide))
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (group, wide)) / torch.where(total == 0, 1.0, total)
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[request, nth])
    s["lse"].copy_((top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[request, nth])


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_gqa_13_gb300 as pd

        pools = (s.get("k"), s.get("v"), s.get("k_scale"), s.get("v_scale"))
        table = (s.get("indices"), s.get("indptr"), s.get("last"))
        if "rot" in c:
            turn = {"layout": pd.PD_ROPE_HALF if c["layout"] == "half" else pd.PD_ROPE_PAIRS, "rope_scale": s["factor"]}
        if op == "rotate":
            pd.pd_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["freqs"], s["q_out"], s["k_out"],
                            EPS, **turn)
        elif op == "append" and c["block"]:
            norm = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS} if c["norm"] else {}
            pd.pd_paged_rope_append_fp8_blocks(s["q"], s["k_new"], s["v_new"], s["positions"], s["freqs"], s["q_out"],
                                               s["k_scale"], s["v_scale"], s["k"], s["v"], *table, s["new_indptr"],
                                               s["workspace"], **norm, **turn)
        elif op == "append":
            pd.pd_paged_norm_rope_append(s["q"], s["k_new"], s["v_new"], s["q_weight"], s["k_weight"], s["positions"],
                                         s["freqs"], s["q_out"], s["k"], s["v"], *table, s["new_indptr"], s["workspace"],
                                         EPS, **turn)
        elif op == "read":
            pd.pd_paged_read_fp8_blocks(*pools, *table, s["new_indptr"], s["first"], s["k_out"], s["v_out"], s["workspace"])
        elif op == "decode":
            pd.pd_paged_decode_fp8_blocks(s["q"], *pools, *table, s["o"], s["lse"], 1 / math.sqrt(c["d"]), s["workspace"])
        else:
            pd.pd_paged_tree_decode_fp8_blocks(s["q"], *pools, *table, s["new_indptr"], s["mask"], s["o"], s["lse"],
                                               1 / math.sqrt(c["d"]), s["workspace"])
    elif op == "rotate":
        s["q_out"].copy_(_rotate(s["q"], s["q_weight"], s["positions"], s))
        s["k_out"].copy_(_rotate(s["k"], s["k_weight"], s["positions"], s))
    else:
        {"append": _plain_append, "read": _plain_read, "decode": _plain_attend, "tree": _plain_attend}[op](s)
    if op == "rotate":
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    if op != "append":
        return {"o": s["o"], "lse": s["lse"]}
    if not c["block"]:
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    k, v = (s[x].view(torch.float8_e4m3fn) for x in ("k", "v"))
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": s["q_out"]}


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, block = case["op"], case.get("block", 0)

    def turned(x, weight, positions):
        """Each head over its norm, each rotated pair as a complex number times factor * exp(i angle)."""
        out = x.double().clone()
        if weight is not None:
            out = out / (out.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * weight.double()
        w = torch.polar(torch.full((positions.numel(), case["rot"] // 2), s["factor"], dtype=torch.float64, device="cuda"),
                        torch.outer(positions.double(), s["inv"]))[:, None]
        h = case["rot"] // 2
        even, odd = (slice(0, h), slice(h, 2 * h)) if case["layout"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
        z = torch.complex(out[..., even], out[..., odd]) * w
        out[..., even], out[..., odd] = z.real, z.imag
        return out

    if op == "rotate":
        return {"q": turned(s["q"], s["q_weight"], s["positions"]), "k": turned(s["k"], s["k_weight"], s["positions"])}
    indices, indptr = s["indices"].cpu().numpy().astype(np.int64), s["indptr"].cpu().numpy()
    start = s["new_indptr"].cpu().numpy()

    def rows(b, tokens):
        return (torch.from_numpy(indices[indptr[b] + tokens // case["page"]]).cuda(),
                torch.from_numpy(tokens % case["page"]).cuda())

    def held(x, b, tokens):
        """[token, head, dim]: what the cache holds."""
        page, row = rows(b, tokens)
        codes, scale = s[x][page, :, row], s[x + "_scale"][page, :, row // block]
        return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]

    if op == "append":
        at = s["positions"]
        if at is None:
            at = torch.from_numpy(np.concatenate([np.arange(l - n, l) for l, n in zip(s["kv"], s["new"])])).cuda()
        weights = (s["q_weight"], s["k_weight"]) if case["norm"] else (None, None)
        fresh = {"k": turned(s["k_new"], weights[1], at), "v": s["v_new"].double()}
        out = {"q": turned(s["q"], weights[0], at)}
        for x in ("k", "v"):
            pool = (s[x].view(torch.float8_e4m3fn) if block else s[x]).double()
            scales = s[x + "_scale"].double() if block else None
            for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
                if n == 0:
                    continue
                new = fresh[x][start[b]:start[b] + n]
                page, row = rows(b, np.arange(l - n, l))
                if not block:
                    pool[page, :, row] = new
                    continue
                first = (l - n) // block * block  # of the request's first block that changes
                lead, tail = l - n - first, -(l - first) % block
                top = torch.nn.functional.pad(new.abs().amax(-1), (0, 0, lead, tail)).unflatten(0, (-1, block)).amax(1)
                bp, br = rows(b, np.arange(first, l, block))
                scale = torch.clamp(top / TOP, min=LEAST)
                if lead:
                    was = scales[bp[0], :, br[0] // block]
                    up = torch.exp2(torch.clamp(torch.ceil(torch.log2(top[0] / (EDGE * was))), min=0.0))
                    scale[0] = was * up
                    op_, or_ = rows(b, np.arange(first, l - n))
                    pool[op_, :, or_] = pool[op_, :, or_] / up[:, None]
                scales[bp, :, br // block] = scale
                each = scale.repeat_interleave(block, 0)[lead:lead + n]
                pool[page, :, row] = (new / each[..., None]).clamp(-TOP, TOP)
            out[x] = pool
            if block:
                out[x + "_scale"] = scales
        return out
    if op == "read":
        k, v = s["k_out"].double(), s["v_out"].double()
        for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
            tokens = np.arange(l - n, l)
            k[start[b]:start[b] + n], v[start[b]:start[b] + n] = held("k", b, tokens), held("v", b, tokens)
        return {"k": k, "v": v}
    group = case["hq"] // case["hk"]
    o, lse = torch.zeros_like(s["o"], dtype=torch.float64), torch.full_like(s["lse"], -math.inf, dtype=torch.float64)
    words = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
        if l == 0 or n == 0:
            continue
        k, v = held("k", b, np.arange(l)), held("v", b, np.arange(l))
        ban = np.zeros((n, l), bool)
        if words is None:
            ban[:, l - n:] = np.triu(np.ones((n, n), bool), 1)
        else:
            j = np.arange(n)
            ban[:, l - n:] = (words[start[b]:start[b] + n][:, j // 32] >> (j % 32).astype(np.uint32)) & 1 == 0
        ban = torch.from_numpy(ban).cuda()
        for h in range(case["hk"]):
            heads = slice(h * group, (h + 1) * group)
            q = s["q"][start[b]:start[b] + n, heads].double().transpose(0, 1)
            x = (q @ k[:, h].T / math.sqrt(case["d"])).masked_fill(ban, -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z))
            o[start[b]:start[b] + n, heads] = (p @ v[:, h]).transpose(0, 1)
            lse[start[b]:start[b] + n, heads] = z[..., 0].T
    return {"o": o, "lse": lse}
