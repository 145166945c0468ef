"""The speculative-decoding operators: cases, plain forms and work.

Four operators that a serving step with drafted tokens chains over one paged
KV cache (pages [num_pages, num_kv_heads, page_size, head_dim], found through
indices / indptr / last_page_len):

- rope: rotary positions applied to the leading rot_dim elements of each head;
- append: new tokens (one, a draft, or a whole prompt per request) rotated and
  written into the pages of their requests, their q rows rotated on the way;
- tree: attention of each request's last rows (drafted nodes, a chain or a
  tree given by a bit mask) over the cached tokens and over each other;
- commit: the accepted nodes' K/V rows moved to the front of the draft.

`run` computes a case either in plain torch operations (own = False) or with
the framework's calls (own = True), on the same state.
"""
import math
import statistics

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
#: One scratch buffer of a serving program, for every call on its stream.
WORKSPACE = 192 << 20


# ---------------------------------------------------------------- cases

def listed():
    base = {"theta": 500000.0, "layout": "half", "scaling": "none"}
    llama = {"hq": 32, "hk": 8, "d": 128, "page": 16}
    seventy = {"hq": 64, "hk": 8, "d": 128, "page": 32}
    return [
        # one decoded token far into a long context: q and k heads of a fused projection
        {"name": "rope_one_token", "op": "rope", "tokens": 1, "heads": 40, "d": 128, "rot": 128, "dtype": "bf16",
         "far": 131071, **base},
        # a prompt of odd length, pairs side by side, half of each head rotated, stretched context
        {"name": "rope_prompt_f16", "op": "rope", "tokens": 8191, "heads": 64, "d": 128, "rot": 64, "dtype": "f16",
         "far": 8191, **base, "layout": "pairs", "scaling": "yarn"},
        # the batched decode step: one token for each of 32 requests of 512 to 4096 tokens
        {"name": "append_b32_bf16", "op": "append", "batch": 32, "new_lo": 1, "new_hi": 1, "kv_lo": 512,
         "kv_hi": 4096, "spread": "uniform", **llama, "rot": 128, "dtype": "bf16", "pool": "bf16",
         "positions": "given", **base, "scaling": "banded"},
        # ragged prompts and drafts together into an E4M3 pool
        {"name": "append_prompts_e4m3", "op": "append", "batch": 24, "new_lo": 1, "new_hi": 4095, "kv_lo": 1,
         "kv_hi": 4095, "spread": "log", **seventy, "rot": 128, "dtype": "f16", "pool": "e4m3",
         "positions": "index", **base, "layout": "pairs"},
        # the smallest call: one request of 100 tokens, 6 nodes, in f32
        {"name": "tree_tiny_f32", "op": "tree", "batch": 1, "new_lo": 6, "new_hi": 6, "kv_lo": 100, "kv_hi": 100,
         "spread": "uniform", "hq": 8, "hk": 2, "d": 64, "page": 16, "dtype": "f32", "pool": "f32", "mask": "tree"},
        # a chain of 4 drafted tokens for each of 32 requests
        {"name": "tree_chain_b32_bf16", "op": "tree", "batch": 32, "new_lo": 4, "new_hi": 4, "kv_lo": 512,
         "kv_hi": 4096, "spread": "uniform", **llama, "dtype": "bf16", "pool": "bf16", "mask": "chain"},
        # a 64-node tree over four long contexts
        {"name": "tree_long_b4_f16", "op": "tree", "batch": 4, "new_lo": 64, "new_hi": 64, "kv_lo": 131072,
         "kv_hi": 131072, "spread": "uniform", **llama, "dtype": "f16", "pool": "f16", "mask": "tree"},
        # trees of 1 to 32 nodes, a large ragged batch over an E4M3 pool, groups of 8 heads
        {"name": "tree_b64_e4m3", "op": "tree", "batch": 64, "new_lo": 1, "new_hi": 32, "kv_lo": 32, "kv_hi": 8192,
         "spread": "lognormal", **seventy, "dtype": "bf16", "pool": "e4m3", "mask": "tree"},
        # no shared heads, head_dim 256
        {"name": "tree_mha_d256_f16", "op": "tree", "batch": 16, "new_lo": 24, "new_hi": 48, "kv_lo": 48,
         "kv_hi": 8191, "spread": "uniform", "hq": 16, "hk": 16, "d": 256, "page": 16, "dtype": "f16", "pool": "f16",
         "mask": "tree"},
        # pieces of four prompts over what is cached of them
        {"name": "tree_chunk_bf16", "op": "tree", "batch": 4, "new_lo": 1021, "new_hi": 1021, "kv_lo": 7000,
         "kv_hi": 8191, "spread": "uniform", **llama, "dtype": "bf16", "pool": "bf16", "mask": "chain"},
        # what 32 requests keep of their 16 nodes
        {"name": "commit_b32_bf16", "op": "commit", "batch": 32, "new_lo": 16, "new_hi": 16, "kv_lo": 512,
         "kv_hi": 4096, "spread": "uniform", **llama, "pool": "bf16", "accept": 5},
        # what 256 requests keep of their 64 nodes, some of them nothing, E4M3 codes
        {"name": "commit_b256_e4m3", "op": "commit", "batch": 256, "new_lo": 24, "new_hi": 64, "kv_lo": 64,
         "kv_hi": 2048, "spread": "log", **seventy, "pool": "e4m3", "accept": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "tree", "tree", "tree", "commit"])
    hq, hk, d, page = rng.choice([(32, 8, 128, 16), (64, 8, 128, 32), (16, 16, 256, 16), (8, 2, 64, 16), (28, 4, 128, 16),
                                  (32, 8, 128, 64), (12, 4, 64, 8)])
    shape = {"hq": hq, "hk": hk, "d": d, "page": page}
    dtype = rng.choice(["f16", "bf16", "bf16"])
    rope = {"rot": rng.choice([d, d, d // 2]), "theta": rng.choice([10000.0, 500000.0]),
            "layout": rng.choice(["half", "pairs"]), "scaling": rng.choice(["none", "linear", "banded", "yarn"])}
    if op == "rope":
        tokens = _log(rng, 1, 8191)
        return {"op": op, "tokens": tokens, "heads": hq + hk, "d": d, "dtype": rng.choice([dtype, dtype, "f32"]),
                "far": max(tokens, _log(rng, 64, 131071)), **rope}
    batch = _log(rng, 1, 64)
    if op == "append":
        hi = _log(rng, 1, max(1, 16384 // batch))
        return {"op": op, "batch": batch, "new_lo": max(1, hi // 4), "new_hi": hi, "kv_lo": hi,
                "kv_hi": hi + _log(rng, 1, 2048), "spread": "uniform", **shape, "dtype": dtype,
                "pool": rng.choice([dtype, dtype, "e4m3"]), "positions": rng.choice(["given", "index"]), **rope}
    if op == "commit":
        hi = _log(rng, 2, 64)
        return {"op": op, "batch": batch, "new_lo": max(1, hi // 2), "new_hi": hi, "kv_lo": hi,
                "kv_hi": hi + _log(rng, 1, 4096), "spread": "log", **shape,
                "pool": rng.choice(["f16", "bf16", "e4m3"]), "accept": rng.randint(1, 12)}
    if rng.random() < 0.12:  # f32: small batches
        hi = _log(rng, 1, 16)
        return {"op": op, "batch": _log(rng, 1, 8), "new_lo": hi, "new_hi": hi, "kv_lo": hi,
                "kv_hi": hi + _log(rng, 16, 4096), "spread": "uniform", **shape, "dtype": "f32", "pool": "f32",
                "mask": rng.choice(["tree", "chain"])}
    mask = rng.choice(["tree", "tree", "chain"])
    hi = _log(rng, 1, 64) if mask == "tree" else _log(rng, 1, 1024)
    tokens = min(131072 * 4 // batch, max(64, int(2.0e11 / (hi * hq * d * 4 * batch))))
    kv = hi + _log(rng, 16, min(131072, tokens))
    return {"op": op, "batch": batch, "new_lo": max(1, hi // 3), "new_hi": hi, "kv_lo": hi + (kv - hi) // 4,
            "kv_hi": kv, "spread": rng.choice(["uniform", "log"]), **shape, "dtype": dtype,
            "pool": rng.choice([dtype, dtype, "e4m3"]), "mask": mask}


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
    w = (np.arange(b) * 0.7548776662466927 + 0.25) % 1.0
    new = np.rint(case["new_lo"] + w * (case["new_hi"] - case["new_lo"])).astype(np.int64)
    return kv, np.minimum(new, kv)


def _accepted_lengths(case, new):
    w = (np.arange(case["batch"]) * 0.5698402909980532 + 0.4) % 1.0
    return np.minimum(np.rint(w * case["accept"]).astype(np.int64), new)


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["d"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    kv, new = _lengths(case)
    pages = int(np.sum(-(-kv // case["page"])))
    table = 4 * (pages + 2 * case["batch"] + 1 + case["batch"] + 1)
    row = case["hk"] * case["d"]
    if op == "append":
        t, e = int(new.sum()), SIZE[case["dtype"]]
        q = case["hq"] * case["d"]
        return {"bytes": t * (2 * q * e + 2 * row * (e + SIZE[case["pool"]])) + table,
                "flops": 3 * t * (case["hq"] + case["hk"]) * case["rot"]}
    if op == "commit":
        kept = int(_accepted_lengths(case, new).sum())
        return {"bytes": 2 * 2 * kept * row * SIZE[case["pool"]] + table + 4 * kept, "flops": 0}
    t = int(new.sum())
    pairs = int(np.sum(new * (kv - new) + (new * (new + 1)) // 2))  # a tree sees fewer of its own nodes
    q = case["hq"] * case["d"]
    return {"bytes": 2 * int(kv.sum()) * row * SIZE[case["pool"]] + 2 * t * q * SIZE[case["dtype"]]
            + 4 * t * case["hq"] + table, "flops": 4 * case["d"] * case["hq"] * pairs}


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


def _pages(kv, page, rng):
    """A shuffled page table over a pool of a tenth more pages than are used."""
    n = -(-kv // page)
    used = int(n.sum())
    total = used + max(1, used // 10)
    indptr = np.concatenate([[0], np.cumsum(n)])
    last = kv - (n - 1) * page
    return rng.permutation(total)[:used], indptr, last, total


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def _normal(shape, dtype, gen):
    if dtype == "e4m3":  # codes of normal values at scale 1 / 64
        return (torch.randn(shape, device="cuda", dtype=torch.float16, generator=gen) * 64).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    return torch.randn(shape, device="cuda", dtype=TYPES[dtype], generator=gen)


def _tree(n, rng):
    """Parents of a drafted tree in breadth-first order: each node hangs from one of the few before it."""
    p = np.arange(n) - 1 - (rng.random(n) * np.minimum(6, np.arange(n) + 1)).astype(np.int64)
    return np.maximum(p, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if "rot" in case:
        inv, factor = _inv_freq(case)
        # the framework's table: each pair's turns per position, in units of 2^-64 turn
        s["freqs"] = torch.from_numpy(np.ldexp(inv / (2 * math.pi), 64).astype(np.uint64).view(np.int64)).cuda()
        s["inv"], s["factor"] = torch.from_numpy(inv).cuda(), factor
    if op == "rope":
        s["x"] = _normal((case["tokens"], case["heads"], case["d"]), case["dtype"], gen)
        first = max(0, case["far"] - case["tokens"] + 1 - int(rng.integers(0, 32)))
        s["positions"] = _i32(first + np.arange(case["tokens"]))
        s["out"] = torch.empty_like(s["x"])
        return s
    kv, new = _lengths(case)
    indices, indptr, last, total = _pages(kv, case["page"], rng)
    s["indices"], s["indptr"], s["last"] = _i32(indices), _i32(indptr), _i32(last)
    starts = np.concatenate([[0], np.cumsum(new)])
    s["new_indptr"] = _i32(starts)
    # on the host, a program knows its requests' lengths
    s["kv"], s["new"] = kv, new
    t = int(new.sum())
    pool = (total, case["hk"], case["page"], case["d"])
    s["k"], s["v"] = _normal(pool, case["pool"], gen), _normal(pool, case["pool"], gen)
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    if case["pool"] == "e4m3":
        s["k_scale"] = torch.rand(case["hk"], device="cuda", generator=gen) * 0.01 + 0.012
        s["v_scale"] = torch.rand(case["hk"], device="cuda", generator=gen) * 0.01 + 0.012
    if op == "append":
        # one projection's output holds q, k and v of a token side by side
        qkv = _normal((t, case["hq"] + 2 * case["hk"], case["d"]), case["dtype"], gen)
        s["q"], s["k_new"], s["v_new"] = (qkv[:, :case["hq"]], qkv[:, case["hq"]:case["hq"] + case["hk"]],
                                          qkv[:, case["hq"] + case["hk"]:])
        s["q_out"] = torch.empty(t, case["hq"], case["d"], dtype=TYPES[case["dtype"]], device="cuda")
        at = np.concatenate([np.arange(n) + (l - n) for l, n in zip(kv, new)])
        s["positions"] = None
        if case["positions"] == "given":
            s["positions"] = _i32(at + 60000)
    elif op == "tree":
        s["q"] = _normal((t, case["hq"], case["d"]), case["dtype"], gen)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(t, case["hq"], device="cuda")
        s["mask"] = None
        if case["mask"] == "tree":
            words = -(-int(new.max()) // 32)
            bits = np.zeros((t, words), np.uint32)
            for b, n in enumerate(new):
                for j, p in enumerate(_tree(int(n), rng)):
                    if p >= 0:
                        bits[starts[b] + j] = bits[starts[b] + p]
                    bits[starts[b] + j, j // 32] |= np.uint32(1 << (j % 32))
            s["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
    else:
        kept = _accepted_lengths(case, new)
        most = max(1, int(kept.max()))
        path = np.full((case["batch"], most), -1, np.int64)
        for b, (n, a) in enumerate(zip(new, kept)):
            # a path down the tree: the first candidate where it was the likeliest, nodes past the kept length otherwise
            free = np.arange(a, n)
            lead = int(a) - len(free) if a > len(free) else int(rng.integers(0, 2)) if a > 0 else 0
            rest = np.sort(rng.choice(free, int(a) - lead, replace=False)) if a > lead else []
            path[b, :a] = np.concatenate([np.arange(lead), rest])
        s["path"], s["path_len"] = _i32(path), _i32(kept)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, positions, inv, factor, rot, layout, wide=torch.float32):
    angle = positions.double()[:, None] * inv
    c, n = (angle.cos() * factor).to(wide)[:, None], (angle.sin() * factor).to(wide)[:, None]
    x = x.to(wide)
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., :rot:2], x[..., 1:rot:2])
    a, b = a * c - b * n, b * c + a * n
    turned = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rows(s, request, token):
    """(page, row) of a request's token."""
    page = s["case"]["page"]
    return s["indices"].long()[s["indptr"].long()[request] + token // page], token % page


def _ragged(s):
    """For each new token: its request, its index among the request's new tokens, its index in the cache."""
    start = s["new_indptr"].long()
    new = start[1:] - start[:-1]
    request = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new, output_size=int(s["new"].sum()))
    nth = torch.arange(request.numel(), device="cuda") - start[request]
    pages = (s["indptr"][1:] - s["indptr"][:-1]).long()
    kv = (pages - 1) * s["case"]["page"] + s["last"].long()
    return request, nth, kv[request] - new[request] + nth, kv, new


def _codes(x, scale):
    return (x / scale.to(x.dtype)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    request, _, token, _, _ = _ragged(s)
    at = token if s["positions"] is None else s["positions"]
    wide = torch.float64 if c["pool"] == "e4m3" else torch.float32  # a code's rounding border is near many values
    turn = (at, s["inv"], s["factor"], c["rot"], c["layout"])
    s["q_out"].copy_(_rotate(s["q"], *turn))
    k, v = _rotate(s["k_new"], *turn, wide), s["v_new"].to(wide)
    if c["pool"] == "e4m3":
        k, v = _codes(k, s["k_scale"]), _codes(v, s["v_scale"])
    page, row = _rows(s, request, token)
    s["k"][page, :, row] = k.to(s["k"].dtype)
    s["v"][page, :, row] = v.to(s["v"].dtype)


def _plain_tree(s):
    c = s["case"]
    request, nth, _, kv, new = _ragged(s)
    most, wide, group = int(s["kv"].max()), int(s["new"].max()), c["hq"] // c["hk"]
    token = torch.arange(most, device="cuda")
    inside = token < kv[:, None]
    page, row = _rows(s, torch.arange(c["batch"], device="cuda")[:, None], torch.where(inside, token, 0))
    k, v = s["k"][page, :, row], s["v"][page, :, row]  # [batch, token, head, dim]
    if c["pool"] == "e4m3":
        k, v = (x.view(torch.float8_e4m3fn).float() * y[:, None] for x, y in ((k, s["k_scale"]), (v, s["v_scale"])))
    k, v = k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)
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


def _plain_commit(s):
    c = s["case"]
    _, _, _, kv, new = _ragged(s)
    first = kv - new
    most = s["path"].shape[1]
    request, nth = torch.nonzero(torch.arange(most, device="cuda") < s["path_len"][:, None], as_tuple=True)
    old = _rows(s, request, first[request] + s["path"].long()[request, nth])
    to = _rows(s, request, first[request] + nth)
    for pool in (s["k"], s["v"]):
        pool[to[0], :, to[1]] = pool[old[0], :, old[1]]


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_gqa_13_gb300 as pd

        fp8 = c.get("pool") == "e4m3"
        scales = (s["k_scale"], s["v_scale"]) if fp8 else ()
        table = (s.get("indices"), s.get("indptr"), s.get("last"), s.get("new_indptr"))
        if "rot" in c:
            turn = {"layout": pd.PD_ROPE_HALF if c["layout"] == "half" else pd.PD_ROPE_PAIRS, "rope_scale": s["factor"]}
        if op == "rope":
            pd.pd_rope(s["x"], s["positions"], s["freqs"], s["out"], **turn)
        elif op == "append":
            call = pd.pd_paged_rope_append_fp8 if fp8 else pd.pd_paged_rope_append
            call(s["q"], s["k_new"], s["v_new"], s["positions"], s["freqs"], s["q_out"], *scales, s["k"], s["v"], *table,
                 s["workspace"], **turn)
        elif op == "tree":
            call = pd.pd_paged_tree_decode_fp8 if fp8 else pd.pd_paged_tree_decode
            call(s["q"], s["k"], s["v"], *scales, *table, s["mask"], s["o"], s["lse"], 1 / math.sqrt(c["d"]),
                 s["workspace"])
        else:
            pd.pd_paged_tree_commit(s["k"], s["v"], *table, s["path"], s["path_len"], s["workspace"])
    elif op == "rope":
        s["out"].copy_(_rotate(s["x"], s["positions"], s["inv"], s["factor"], c["rot"], c["layout"]))
    else:
        {"append": _plain_append, "tree": _plain_tree, "commit": _plain_commit}[op](s)
    if op == "rope":
        return s["out"]
    if op == "tree":
        return {"o": s["o"], "lse": s["lse"]}
    k, v = (x.view(torch.float8_e4m3fn) if c["pool"] == "e4m3" else x for x in (s["k"], s["v"]))
    return {"k": k, "v": v, "q": s["q_out"]} if op == "append" else {"k": k, "v": v}


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def turned(x, positions):
        """Each rotated pair as a complex number times factor * exp(i angle)."""
        w = torch.polar(torch.full((positions.numel(), case["rot"] // 2), s["factor"], dtype=torch.float64, device="cuda"),
                        torch.outer(positions.double(), s["inv"]))[:, None]
        out = x.double().clone()
        h = case["rot"] // 2
        even, odd = (slice(0, h), slice(h, 2 * h)) if case["layout"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
        z = torch.complex(out[..., even], out[..., odd]) * w
        out[..., even], out[..., odd] = z.real, z.imag
        return out

    if op == "rope":
        return turned(s["x"], s["positions"])
    indices, indptr = s["indices"].cpu().numpy().astype(np.int64), s["indptr"].cpu().numpy()
    start = s["new_indptr"].cpu().numpy()
    fp8 = case["pool"] == "e4m3"

    def value(codes):
        return (codes.view(torch.float8_e4m3fn) if fp8 else codes).double()

    def rows(b, tokens):
        return (torch.from_numpy(indices[indptr[b] + tokens // case["page"]]).cuda(),
                torch.from_numpy(tokens % case["page"]).cuda())

    if op == "append":
        k, v = value(s["k"]), value(s["v"])
        at = s["positions"]
        if at is None:
            at = torch.from_numpy(np.concatenate([np.arange(l - n, l) for l, n in zip(s["kv"], s["new"])])).cuda()
        q, kn, vn = turned(s["q"], at), turned(s["k_new"], at), s["v_new"].double()
        if fp8:
            kn, vn = ((x / y.double()[:, None]).clamp(-448, 448) for x, y in ((kn, s["k_scale"]), (vn, s["v_scale"])))
        for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
            page, row = rows(b, np.arange(l - n, l))
            k[page, :, row], v[page, :, row] = kn[start[b]:start[b] + n], vn[start[b]:start[b] + n]
        return {"k": k, "v": v, "q": q}
    if op == "commit":
        k, v = value(s["k"]), value(s["v"])
        path, kept = s["path"].cpu().numpy(), s["path_len"].cpu().numpy()
        for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
            old, to = rows(b, l - n + path[b, :kept[b]].astype(np.int64)), rows(b, l - n + np.arange(kept[b]))
            for pool, x in ((k, s["k"]), (v, s["v"])):
                pool[to[0], :, to[1]] = value(x[old[0], :, old[1]])
        return {"k": k, "v": v}
    group = case["hq"] // case["hk"]
    o, lse = s["o"].double(), s["lse"].double()
    words = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b, (l, n) in enumerate(zip(s["kv"], s["new"])):
        page, row = rows(b, np.arange(l))
        k, v = value(s["k"][page, :, row]), value(s["v"][page, :, row])
        if fp8:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
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
