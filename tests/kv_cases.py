"""Inputs of the key-value cache tests: pools, page tables and trees from a seed, on the CPU."""
import dataclasses

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def random_tree(rng, n: int, deepest: int = 8):
    """(parent, depth) of n nodes in canonical order."""
    parent, depth = np.full(n, -1, np.int32), np.zeros(n, np.int32)
    for i in range(1, n):
        lo = max(0, i - 9)
        at = rng.randint(lo, i)
        while depth[at] >= deepest:
            at = parent[at]
        parent[i], depth[i] = at, depth[at] + 1
    order = np.argsort(depth, kind="stable")
    back = np.empty(n, np.int64)
    back[order] = np.arange(n)
    p = parent[order]
    return np.where(p < 0, -1, back[p]).astype(np.int32), depth[order].astype(np.int32)


@dataclasses.dataclass
class Case:
    dtype: torch.dtype
    k: torch.Tensor           # [layers][pages][page][Hkv][D], possibly a transposed view
    v: torch.Tensor
    table: torch.Tensor
    seq_len: torch.Tensor
    parent: object            # int32 [B][nodes] or None
    depth: object
    n_nodes: object
    counts: list
    begin: int
    N: int

    def pools(self, layer):
        """Float64 copies of one layer's pools."""
        return self.k[layer].double().numpy(), self.v[layer].double().numpy()


def make(seed, lens, N, Hkv, D, page, dtype="bf16", tree=True, begin=0, counts=None, layers=1, layout="token",
         stale=0.0, spare=2):
    """Slots that hold no token or node carry `stale` (NaN, infinity, ...), as do the spare pages."""
    rng = np.random.RandomState(seed)
    B, total = len(lens), begin + N
    per = [-(-(int(t) + total) // page) for t in lens]
    pages = sum(per) + spare
    table = np.full((B, max(per) + 1), -1, np.int32)
    perm, at = rng.permutation(pages), 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
    live = [total] * B if counts is None else counts
    pools = []
    for _ in range(2):
        x = torch.full((layers, pages, page, Hkv, D), stale, dtype=DT[dtype])
        for b in range(B):
            for s in range(int(lens[b]) + min(live[b], total)):
                x[:, int(table[b, s // page]), s % page] = torch.from_numpy(rng.standard_normal((layers, Hkv, D))).to(DT[dtype])
        pools.append(x.transpose(2, 3).contiguous().transpose(2, 3) if layout == "head" else x)
    parent = depth = None
    if tree:
        trees = [random_tree(rng, total) for _ in range(B)]
        parent = torch.from_numpy(np.stack([t[0] for t in trees]))
        depth = torch.from_numpy(np.stack([t[1] for t in trees]))
        for b in range(B):
            parent[b, live[b]:] = -1
            depth[b, live[b]:] = -1
    return Case(DT[dtype], pools[0], pools[1], torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32), parent,
                depth, None if counts is None else torch.tensor(counts, dtype=torch.int32), live, begin, N)


def half_step(dtype):
    """Half a rounding step relative to the value: 2^-8 for bf16, 2^-11 for f16."""
    return torch.finfo(dtype).eps / 2


def attend_bound(dtype, out, mean_abs, score_abs, sum_abs, D, tokens):
    """|error| of an attention output: the weights are rounded to dtype (half a step of sum p |v|), scores are
    float32 sums of D products (D + 8 half steps 2^-23 of sum |q k|, twice in the ratio of weights), sums over
    the tokens and the exponential cost (tokens + 16) 2^-23, f16 weights below 2^-14 lose at most 2^-25 each;
    then the output is rounded once."""
    h = half_step(dtype)
    delta = h + 2 * (D + 8) * 2.0 ** -23 * score_abs[..., None] + (tokens + 16) * 2.0 ** -23
    before = delta * (1 + delta) * mean_abs + (2.0 ** -25 * sum_abs if dtype == torch.float16 else 0.0)
    return before + h * (np.abs(out) + before) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
