"""One layer's share of a serving loop with drafted tokens, through the library's calls.

A prompt goes into the paged cache as a chain (rotated append, tree decode without a mask). Then every step drafts a
tree of tokens, appends it, attends for all of its nodes at once, accepts a path, and keeps that path's rows. The host
owns the page table, as with every call of the library. At the end the cache must hold what a plain token-by-token
append of the accepted tokens holds.

    python examples/speculative_step.py
"""
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import paged_kv_gqa_13_gb300 as pd  # noqa: E402

HQ, HK, D, PAGE = 32, 8, 128, 16


class Table:
    """The host's page table: the pages and length of every request over one free list."""

    def __init__(self, batch, pages):
        self.free = list(range(pages))[::-1]
        self.pages = [[] for _ in range(batch)]
        self.length = [0] * batch

    def grow(self, b, n):
        self.length[b] += n
        while len(self.pages[b]) * PAGE < self.length[b]:
            self.pages[b].append(self.free.pop())

    def shrink(self, b, n):
        self.length[b] -= n
        while len(self.pages[b]) > max(1, -(-self.length[b] // PAGE)):
            self.free.append(self.pages[b].pop())

    def device(self, new):
        """indices, indptr, last_page_len, new_indptr for `new` new rows of each request."""
        last = [n - (len(p) - 1) * PAGE for n, p in zip(self.length, self.pages)]
        arrays = (sum(self.pages, []), np.cumsum([0] + [len(p) for p in self.pages]), last, np.cumsum([0] + list(new)))
        return tuple(torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in arrays)


def draft(rng, n):
    """Parents of a tree in breadth-first order (-1: hangs from the last accepted token), depths, and its mask words."""
    parent = np.array([int(rng.integers(max(-1, j - 4), j)) for j in range(n)])
    depth = np.zeros(n, np.int64)
    bits = np.zeros((n, -(-n // 32)), np.uint32)
    for j, p in enumerate(parent):
        if p >= 0:
            depth[j], bits[j] = depth[p] + 1, bits[p]
        bits[j, j // 32] |= np.uint32(1 << (j % 32))
    return parent, depth, bits


def main(batch=4, prompt=300, steps=6, nodes=12, seed=0, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    freqs, rope_scale = pd.pd_rope_frequencies(D, 500000.0, pd.PD_ROPE_BANDED, 8.0)
    pages = batch * (-(-(prompt + steps * (nodes + 2)) // PAGE) + 1)
    k = torch.zeros(pages, HK, PAGE, D, dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    table = Table(batch, pages)
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(HQ, HK, D, pd.PD_BF16))
    kept = [[] for _ in range(batch)]  # the (k, v) rows of the accepted tokens, unrotated

    def step(qkv, new, positions, mask):
        """Append qkv's new rows and attend for them; the table already holds them."""
        t = qkv.shape[0]
        dev = table.device(new)
        q = torch.empty(t, HQ, D, dtype=dtype, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(t, HQ, device="cuda")
        pd.pd_paged_rope_append(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], positions, freqs, q, k, v, *dev, ws,
                                rope_scale=rope_scale)
        pd.pd_paged_tree_decode(q, k, v, *dev, mask, o, lse, 1 / math.sqrt(D), ws)
        return o, dev

    def rows(n):
        return torch.randn(n, HQ + 2 * HK, D, dtype=dtype, device="cuda", generator=gen)

    # the prompts, of different lengths, as chains
    lengths = [prompt - 7 * b for b in range(batch)]
    for b, n in enumerate(lengths):
        table.grow(b, n)
    qkv = rows(sum(lengths))
    step(qkv, lengths, None, None)
    at = np.cumsum([0] + lengths)
    for b in range(batch):
        kept[b].append(qkv[at[b]:at[b + 1], HQ:])

    for _ in range(steps):
        trees = [draft(rng, nodes) for _ in range(batch)]
        before = list(table.length)
        for b in range(batch):
            table.grow(b, nodes)
        qkv = rows(batch * nodes)
        positions = np.concatenate([before[b] + trees[b][1] for b in range(batch)])
        mask = torch.from_numpy(np.concatenate([t[2] for t in trees]).view(np.int32)).cuda()
        o, dev = step(qkv, [nodes] * batch, torch.from_numpy(positions.astype(np.int32)).cuda(), mask)
        # accept the path to the node whose output's first element is largest (a stand-in for the verifier)
        best = o.view(batch, nodes, HQ, D)[:, :, 0, 0].argmax(1).tolist()
        path = np.full((batch, nodes), -1, np.int32)
        accepted = []
        for b in range(batch):
            way, j = [], best[b]
            while j >= 0:
                way.append(j)
                j = int(trees[b][0][j])
            accepted.append(way[::-1])
            path[b, :len(way)] = way[::-1]
            kept[b].append(qkv[b * nodes:(b + 1) * nodes, HQ:][way[::-1]])
        lens = torch.tensor([len(x) for x in accepted], dtype=torch.int32, device="cuda")
        pd.pd_paged_tree_commit(k, v, *dev, torch.from_numpy(path).cuda(), lens, ws, total_new=batch * nodes)
        for b in range(batch):
            table.shrink(b, nodes - len(accepted[b]))
    flags = pd.pd_read_device_flags(ws)

    # the same tokens appended plainly, into a cache of their own
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    new = torch.cat([torch.cat(x) for x in kept])
    pd.pd_paged_rope_append(None, new[:, :HK], new[:, HK:], None, freqs, None, k2, v2, *table.device(table.length), ws,
                            rope_scale=rope_scale)
    same = True
    for b in range(batch):
        tokens = torch.arange(table.length[b], device="cuda")
        page = torch.tensor(table.pages[b], device="cuda")[tokens // PAGE]
        same &= bool(torch.equal(k[page, :, tokens % PAGE], k2[page, :, tokens % PAGE]))
        same &= bool(torch.equal(v[page, :, tokens % PAGE], v2[page, :, tokens % PAGE]))
    return flags, same, table.length


if __name__ == "__main__":
    flags, same, length = main()
    print(f"status word {flags}, the cache is the plain one: {same}, tokens per request {length}")
    sys.exit(0 if flags == 0 and same else 1)
