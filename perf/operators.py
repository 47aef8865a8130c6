"""Work of the target-model operators: the paged key-value cache that a speculative tree is appended to, the
attention of the tree's nodes over it, and the commit of the accepted path.

  append   keys and values of a tree's nodes (optionally normalised per head) rotated to their positions and
           written to the pages of their sequence; the queries normalised and rotated alongside
  attend   every node of the tree attends to the committed tokens of its sequence and to its own ancestors;
           one node is ordinary decoding, a chain of nodes a chunk of a prompt
  commit   after verification, the accepted nodes' keys and values moved to follow the committed tokens,
           in every layer

The trees are those of the framework's workloads (R = 60 nodes and the root, depth 8; 32 nodes at depth 6;
frontiers of 8), the caches generic: 16 to 128 tokens a page, heads of 64 or 128.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 500000.0


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one token of one sequence: the latency of a plain decoding step
        dict(name="append_one", op="append", dtype="bf16", B=1, N=1, begin=0, tree=False, Hq=32, Hkv=8, D=128,
             page=16, length=700, norm=False, rot=128, interleaved=False, layout="token"),
        # a batch of 64 trees of 61 nodes with normalised heads: the verification step's append
        dict(name="append_tree_b64", op="append", dtype="bf16", B=64, N=61, begin=0, tree=True, Hq=32, Hkv=8, D=128,
             page=16, length=1024, norm=True, rot=128, interleaved=False, layout="token"),
        # one short sequence, one token: latency of the attention alone
        dict(name="one_b1_short", op="attend", dtype="bf16", B=1, N=1, begin=0, tree=False, Hq=32, Hkv=8, D=128,
             page=16, length=500, layout="token"),
        # a decoding batch with ragged contexts around 4000 tokens: bandwidth
        dict(name="one_b64", op="attend", dtype="bf16", B=64, N=1, begin=0, tree=False, Hq=32, Hkv=8, D=128,
             page=16, length=5000, layout="token"),
        # two very long contexts: the cache's length has to be split over the card
        dict(name="one_long", op="attend", dtype="bf16", B=2, N=1, begin=0, tree=False, Hq=32, Hkv=8, D=128,
             page=64, length=131071, layout="head"),
        # verification of 8 trees of 61 nodes over ordinary contexts
        dict(name="tree_b8", op="attend", dtype="bf16", B=8, N=61, begin=0, tree=True, Hq=32, Hkv=8, D=128,
             page=16, length=2300, layout="token"),
        # the same for 64 trees: the largest verification step
        dict(name="tree_b64", op="attend", dtype="bf16", B=64, N=61, begin=0, tree=True, Hq=32, Hkv=8, D=128,
             page=32, length=4500, layout="token"),
        # a model with as many key heads as query heads, in half precision
        dict(name="tree_mha_f16", op="attend", dtype="f16", B=6, N=61, begin=0, tree=True, Hq=32, Hkv=32, D=128,
             page=16, length=1500, layout="token"),
        # a drafter's frontier of 8 nodes behind 25 earlier ones, narrow heads
        dict(name="frontier_d64", op="attend", dtype="bf16", B=64, N=8, begin=25, tree=True, Hq=16, Hkv=4, D=64,
             page=32, length=2048, layout="head"),
        # a chunk of a prompt behind an earlier part: long rows of queries, bound by the tensor cores
        dict(name="chunk_2k", op="attend", dtype="bf16", B=1, N=2048, begin=0, tree=False, Hq=32, Hkv=8, D=128,
             page=128, length=2100, layout="token"),
        # the accepted path of one tree in one layer
        dict(name="commit_one", op="commit", dtype="bf16", B=1, N=61, depth=8, layers=1, Hkv=8, D=128, page=16,
             length=600, layout="token"),
        # 16 trees, all 32 layers of the model
        dict(name="commit_b16", op="commit", dtype="bf16", B=16, N=61, depth=8, layers=32, Hkv=8, D=128, page=16,
             length=400, layout="token"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "commit"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), D=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), layout=rng.choice(["token", "head"]))
    if op == "commit":
        c.update(B=_log(rng, 1, 16), N=rng.choice([33, 61, rng.randint(2, 61)]), depth=rng.choice([6, 8]),
                 layers=_log(rng, 1, 32), Hkv=rng.choice([1, 4, 8]), length=_log(rng, 1, 400))
        return c
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 4, 5, 7, 8])
    kind = rng.choice(["one", "one", "tree", "tree", "frontier", "chunk"])
    c.update(Hq=hkv * group, Hkv=hkv, begin=0, tree=kind in ("tree", "frontier"))
    if kind == "one":
        c.update(N=1, B=_log(rng, 1, 64))
    elif kind == "tree":
        c.update(N=rng.choice([33, 61, rng.randint(2, 128)]), B=_log(rng, 1, 48))
    elif kind == "frontier":
        c.update(N=rng.choice([6, 8]), begin=rng.randint(1, 49), B=_log(rng, 1, 64))
    else:
        c.update(N=_log(rng, 17, 1500), B=1)
    if op == "append":
        c.update(length=_log(rng, 1, 1000), norm=rng.random() < 0.5, rot=rng.choice([c["D"], c["D"], c["D"] // 2]),
                 interleaved=rng.random() < 0.3)
        return c
    # keep the cache under about 2 GB and the products under the largest case's
    most = min(131072, int(2.5e5 * 8 * 128 / (c["B"] * hkv * c["D"])), int(2.0e11 / (4.0 * c["B"] * c["N"] * c["Hq"] * c["D"])))
    c["length"] = _log(rng, 1, max(2, most))
    return c


# ------------------------------------------------------------------ inputs ---

def _lengths(case):
    """Committed tokens per sequence, from the case alone: ragged, the longest of `length` tokens."""
    r = np.random.RandomState(case["length"] * 131 + case["B"])
    n = np.maximum(1, (case["length"] * (0.6 + 0.4 * r.rand(case["B"]))).astype(np.int64))
    n[0] = case["length"]
    return n


def _trees(case):
    """(parent, depth, n_nodes) of random trees in canonical order (depth ascending), -1 past n_nodes."""
    B, total = case["B"], case.get("begin", 0) + case["N"]
    deepest = case.get("depth", 8)
    r = np.random.RandomState(total * 977 + B)
    parent = np.full((B, total), -1, np.int32)
    depth = np.full((B, total), -1, np.int32)
    n_nodes = np.zeros(B, np.int32)
    for b in range(B):
        n = total if b % 4 != 3 else max(1, total - r.randint(0, max(1, total // 4)))  # some trees end early
        d = np.concatenate([[0], np.sort(np.minimum(np.arange(n - 1) % deepest, r.randint(0, deepest, n - 1)) + 1)]) if n > 1 else np.zeros(1, np.int64)
        d = np.concatenate([[0], 1 + np.unique(d[1:], return_inverse=True)[1]]).astype(np.int64) if n > 1 else d
        for i in range(1, n):
            above = np.flatnonzero(d[:i] == d[i] - 1)
            parent[b, i] = above[r.randint(len(above))]
        depth[b, :n] = d
        n_nodes[b] = n
    return parent, depth, n_nodes


def _paths(case, parent, n_nodes, seed):
    """An accepted path per tree: a walk from the root down, -1 behind it."""
    r = np.random.RandomState(seed % (1 << 31))
    out = np.full((case["B"], case["depth"] + 1), -1, np.int32)
    acc = np.zeros(case["B"], np.int32)
    for b in range(case["B"]):
        at = 0
        for j in range(case["depth"]):
            kids = np.flatnonzero(parent[b, 1:n_nodes[b]] == at) + 1
            if not len(kids) or r.rand() < 0.08:
                break
            at = kids[r.randint(len(kids))]
            out[b, j] = at
            acc[b] += 1
    return out, acc


def _pool(case, tokens, gen, layers=1):
    """K and V pools [layers][pages][page][Hkv][D] (or heads before tokens), and the page table."""
    page, B = case["page"], case["B"]
    per = [-(-int(t) // page) for t in tokens]
    width, pages = max(per), sum(per) + 3
    r = np.random.RandomState(gen.initial_seed() % (1 << 31))
    perm = r.permutation(pages)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
    shape = (layers, pages, page, case["Hkv"], case["D"]) if case["layout"] == "token" else (layers, pages, case["Hkv"], page, case["D"])
    kv = [torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if layers == 1 else DT[case["dtype"]]).to(DT[case["dtype"]]) for _ in range(2)]
    if case["layout"] == "head":
        kv = [x.transpose(2, 3) for x in kv]
    return kv[0], kv[1], torch.from_numpy(table).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 11)
    dt, B, N, D, Hkv = DT[case["dtype"]], case["B"], case["N"], case["D"], case["Hkv"]
    lens = _lengths(case)
    total = case.get("begin", 0) + N
    s = dict(case=case, seq_len=torch.from_numpy(lens.astype(np.int32)).cuda())
    if case["op"] == "commit" or case["tree"]:
        parent, depth, n_nodes = _trees(case)
        s.update(parent=torch.from_numpy(parent).cuda(), depth=torch.from_numpy(depth).cuda(), n_nodes=torch.from_numpy(n_nodes).cuda())
    else:
        s.update(parent=None, depth=None, n_nodes=None)
    s["k"], s["v"], s["table"] = _pool(case, lens + total, gen, case.get("layers", 1))

    def normal(*shape, gain=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * gain).to(dt)

    if case["op"] == "commit":
        out_node, acc = _paths(case, parent, n_nodes, seed)
        s.update(out_node=torch.from_numpy(out_node).cuda(), accept_len=torch.from_numpy(acc).cuda(), new_len=torch.zeros(B, dtype=torch.int32, device="cuda"))
    elif case["op"] == "append":
        # the projection's output as a model has it: queries, keys and values of a token side by side
        qkv = normal(B, N, case["Hq"] + 2 * Hkv, D)
        s["q_in"], s["k_in"], s["v_in"] = qkv[:, :, :case["Hq"]], qkv[:, :, case["Hq"]:case["Hq"] + Hkv], qkv[:, :, case["Hq"] + Hkv:]
        s["q_out"] = torch.zeros((B, N, case["Hq"], D), dtype=dt, device="cuda")
        s["qw"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt) if case["norm"] else None
        s["kw"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt) if case["norm"] else None
        half = case["rot"] // 2
        ang = torch.arange(int(lens.max()) + total, dtype=torch.float64, device="cuda")[:, None] * THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    else:
        s["q"] = normal(B, N, case["Hq"], D, gain=1.5)
        s["out"] = torch.zeros((B, N, case["Hq"], D), dtype=dt, device="cuda")
    if own:
        from dynamic_tree_speculative_gb300 import binding as F
        s["cache"] = F.KVCache(s["k"], s["v"], s["table"], s["seq_len"])
        s["nodes"] = F.NodeArrays(s["parent"], s["depth"], s["n_nodes"]) if s["parent"] is not None else None
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "attend":
            s["workspace"] = F.AttendWorkspace(B, N, case["Hq"], Hkv, D)
    return s


# --------------------------------------------------------------- one pass ---

def run(s):
    return {"append": _append, "attend": _attend, "commit": _commit}[s["case"]["op"]](s)


def _slots(s, node):
    """(page, offset) of tree node `node` [B, n] of every sequence."""
    pos = s["seq_len"].long()[:, None] + node
    page = s["case"]["page"]
    return torch.gather(s["table"].long(), 1, (pos // page).clamp(0, s["table"].shape[1] - 1)), pos % page


def _live(s):
    """Truth values [B, N]: the query's node belongs to its tree."""
    c = s["case"]
    node = c["begin"] + torch.arange(c["N"], device="cuda")
    return (node[None] < s["n_nodes"][:, None]) if s["n_nodes"] is not None else torch.ones((c["B"], c["N"]), dtype=torch.bool, device="cuda")


def _append(s):
    c = s["case"]
    if own:
        from dynamic_tree_speculative_gb300 import binding as F
        F.spec_tree_kv_append(s["cache"], 0, s["q_in"], s["k_in"], s["v_in"], s["q_out"], s["rope"], s["status"],
                              tree=s["nodes"], node_begin=c["begin"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    node = c["begin"] + torch.arange(c["N"], device="cuda")
    depth = s["depth"][:, c["begin"]:].long() if s["depth"] is not None else node[None].expand(c["B"], -1)
    table = s["rope"][(s["seq_len"].long()[:, None] + depth).clamp_min(0)][:, :, None]
    half = c["rot"] // 2
    cos, sin = table[..., :half], table[..., half:]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([r, rest], -1).to(s["q_out"].dtype)

    live = _live(s)
    s["q_out"].copy_(torch.where(live[:, :, None, None], turned(s["q_in"], s["qw"]), 0))
    page, off = _slots(s, node[None].expand(c["B"], -1))
    s["k"][0].index_put_((page[live], off[live]), turned(s["k_in"], s["kw"])[live])
    s["v"][0].index_put_((page[live], off[live]), s["v_in"][live])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _attend(s):
    c = s["case"]
    if own:
        from dynamic_tree_speculative_gb300 import binding as F
        F.spec_tree_attend(s["cache"], 0, s["q"], s["out"], s["workspace"], s["status"], tree=s["nodes"], node_begin=c["begin"])
        return s["out"]
    B, N, Hq, Hkv, D, page = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
    total = c["begin"] + N
    longest = min(c["length"] + total, s["table"].shape[1] * page)
    at = torch.arange(longest, device="cuda")
    pages = s["table"].long().clamp_min(0)[:, at // page]
    k = s["k"][0][pages, at % page].float()  # [B, tokens, Hkv, D]
    v = s["v"][0][pages, at % page].float()
    node = at[None] - s["seq_len"].long()[:, None]  # the tree node that a token is, negative for committed ones
    if s["parent"] is not None:
        up = torch.nn.functional.one_hot(s["parent"].long() + 1, total + 1)[..., 1:].double()
        sees = torch.linalg.matrix_power(up + torch.eye(total, dtype=torch.float64, device="cuda"), total) > 0
        sees = sees[:, c["begin"]:] & _live(s)[:, :, None]
    else:
        sees = torch.ones((total, total), dtype=torch.bool, device="cuda").tril()[c["begin"]:].expand(B, -1, -1)
    mask = torch.gather(sees, 2, node.clamp(0, total - 1)[:, None].expand(-1, N, -1))
    mask = ((node[:, None] < 0) | (mask & (node[:, None] < total))) & _live(s)[:, :, None]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, N, longest) / math.sqrt(D)
    score = score.masked_fill_(~mask[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = score.sub_(top).exp_()
    total_p = p.sum(-1, keepdim=True)
    v = v.masked_fill((at[None] >= s["seq_len"].long()[:, None] + total)[:, :, None, None], 0)
    o = (p.view(B, Hkv, -1, longest) @ v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, N, D) / total_p.clamp_min(1e-30)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D))
    return s["out"]


def _commit(s):
    c = s["case"]
    if own:
        from dynamic_tree_speculative_gb300 import binding as F
        F.spec_tree_kv_commit(s["cache"], s["accept_len"], s["out_node"], s["new_len"], s["status"])
        return {"k": s["k"], "v": s["v"], "new_len": s["new_len"]}
    step = torch.arange(c["depth"], device="cuda")
    taken = step[None] < s["accept_len"][:, None]
    src = _slots(s, s["out_node"][:, :c["depth"]].long().clamp_min(0))
    dst = _slots(s, (step + 1)[None].expand(c["B"], -1))
    for x in (s["k"], s["v"]):
        x[:, dst[0][taken], dst[1][taken]] = x[:, src[0][taken], src[1][taken]]
    s["new_len"].copy_(s["seq_len"] + 1 + s["accept_len"])
    return {"k": s["k"], "v": s["v"], "new_len": s["new_len"]}


# -------------------------------------------------------- what a pass costs ---

def work(case):
    lens, size = _lengths(case).astype(float), 2
    D, Hkv, B, N = case["D"], case["Hkv"], case["B"], case["N"]
    parent, depth, n_nodes = _trees(case) if case["op"] == "commit" or case["tree"] else (None, None, None)
    total = case.get("begin", 0) + N
    live = np.clip((n_nodes if n_nodes is not None else np.full(B, total)) - case.get("begin", 0), 0, N)
    if case["op"] == "commit":
        _, acc = _paths(case, parent, n_nodes, 1)
        return {"bytes": float(2 * acc.sum() * 2 * case["layers"] * Hkv * D * size + 8 * B), "flops": 0.0}
    if case["op"] == "append":
        row = (case["Hq"] + 2 * Hkv) * D
        return {"bytes": float(live.sum() * (2 * row * size + 4 * case["rot"])), "flops": float(live.sum() * row * (6 + 4 * case["norm"]))}
    tokens = lens + (n_nodes if n_nodes is not None else total)
    if case["tree"]:
        d = depth[:, case["begin"]:]
        seen = float(sum((live[b] * lens[b]) + (d[b][d[b] >= 0] + 1).sum() for b in range(B)))
    else:
        seen = float((N * lens + N * case["begin"] + N * (N + 1) / 2).sum())
    return {"bytes": float(tokens.sum() * 2 * Hkv * D * size + 2 * live.sum() * case["Hq"] * D * size), "flops": 4.0 * seen * case["Hq"] * D}


# ----------------------------------------------------- the definition in 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, "cuda"
    B, page, D = c["B"], c["page"], c["D"]
    lens, table = s["seq_len"].tolist(), s["table"].cpu().numpy()
    if c["op"] == "commit":
        # a copy: the values are the cache's own
        nodes, acc = s["out_node"].tolist(), s["accept_len"].tolist()
        k, v = s["k"], s["v"]
        for b in range(B):
            ids = nodes[b][:acc[b]]
            place = lambda n: (int(table[b, (lens[b] + n) // page]), (lens[b] + n) % page)  # noqa: E731
            held = [(k[:, place(n)[0], place(n)[1]].clone(), v[:, place(n)[0], place(n)[1]].clone()) for n in ids]
            for j, (hk, hv) in enumerate(held):
                p, o = place(j + 1)
                k[:, p, o], v[:, p, o] = hk, hv
        return {"k": k, "v": v, "new_len": torch.tensor([lens[b] + 1 + acc[b] for b in range(B)], dtype=torch.int32)}
    begin, N = c["begin"], c["N"]
    counts = s["n_nodes"].tolist() if s["n_nodes"] is not None else [begin + N] * B
    if c["op"] == "append":
        half, rot = c["rot"] // 2, c["rot"]
        q = torch.zeros((B, N, c["Hq"], D), dtype=torch.float64, device=dev)
        k, v = s["k"].double(), s["v"].double()
        depth = s["depth"].cpu().numpy() if s["depth"] is not None else None
        idx = torch.arange(D, device=dev)
        # element i of a turned vector is x_i cos + x_partner sin, the first of a pair with a minus
        if c["interleaved"]:
            first, pair, freq = idx % 2 == 0, torch.where(idx % 2 == 0, idx + 1, idx - 1), idx // 2
        else:
            first, pair, freq = idx < half, torch.where(idx < half, idx + half, idx - half), idx % half
        turns = idx < rot
        freq, pair = torch.where(turns, freq, 0), torch.where(turns, pair, idx)
        for b in range(B):
            n = max(0, min(N, counts[b] - begin))
            if not n:
                continue
            steps = depth[b, begin:begin + n] if depth is not None else np.arange(begin, begin + n)
            rows = s["rope"].double()[torch.from_numpy(np.asarray(steps, np.int64) + lens[b]).to(dev)]
            cos = torch.where(turns, rows[:, freq], 1.0)[:, None]
            sin = torch.where(turns, torch.where(first, -rows[:, half + freq], rows[:, half + freq]), 0.0)[:, None]
            made = []
            for x, w in ((s["q_in"], s["qw"]), (s["k_in"], s["kw"])):
                x = x[b, :n].double()
                if w is not None:
                    x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
                made.append(x * cos + x[..., pair] * sin)
            q[b, :n] = made[0]
            where = np.arange(begin, begin + n) + lens[b]
            pg, off = torch.from_numpy(table[b, where // page].astype(np.int64)).to(dev), torch.from_numpy(where % page).to(dev)
            k[0, pg, off], v[0, pg, off] = made[1], s["v_in"][b, :n].double()
        return {"q": q, "k": k, "v": v}
    group = c["Hq"] // c["Hkv"]
    out = torch.zeros((B, N, c["Hq"], D), dtype=torch.float64, device=dev)
    parent = s["parent"].cpu().numpy() if s["parent"] is not None else None
    for b in range(B):
        n = max(0, min(N, counts[b] - begin))
        if not n:
            continue
        tokens = lens[b] + counts[b]
        where = np.arange(tokens)
        pg, off = torch.from_numpy(table[b, where // page].astype(np.int64)).to(dev), torch.from_numpy(where % page).to(dev)
        sees = np.zeros((n, counts[b]), bool)
        for i in range(n):
            if parent is None:
                sees[i, :begin + i + 1] = True
            else:
                at = begin + i
                while at >= 0:
                    sees[i, at] = True
                    at = parent[b, at]
        hidden = torch.from_numpy(~sees).to(dev)
        for h in range(c["Hkv"]):
            kh, vh = s["k"][0, pg, off, h].double(), s["v"][0, pg, off, h].double()
            for g in range(group):
                x = s["q"][b, :n, h * group + g].double() @ kh.T * D ** -0.5
                x[:, lens[b]:][hidden] = -math.inf
                out[b, :n, h * group + g] = torch.softmax(x, -1) @ vh
    return out
