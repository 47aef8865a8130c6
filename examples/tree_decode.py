#!/usr/bin/env python
"""Speculative decoding of a batch with dynamic trees, end to end on one GPU.

A small transformer with random weights stands in for the target model and a
one-layer one for the drafter; everything that the framework provides runs as it
would around real ones:

  drafting      the drafter runs on each frontier (spec_tree_kv_append and
                spec_tree_attend with the frontier's parents), spec_tree_layer
                expands it, spec_tree_finish prunes the tree
  verification  the target runs over all nodes of the tree at once
                (spec_tree_kv_append, spec_tree_attend with the tree's parents),
                spec_tree_verify accepts a path and draws the bonus token
  commit        spec_tree_kv_commit moves the accepted path's keys and values
                behind the committed tokens; the drafter appends them as a chain

With --bits 4 both models keep their keys and values in 4 bits (the spec_tree_kv4_*
calls), in pages that a pool hands out as sequences grow and takes back from the
nodes that were not accepted (spec_tree_kv_reserve, spec_tree_kv_release).

    python examples/tree_decode.py [--rounds 12] [--batch 4] [--bits 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dynamic_tree_speculative_gb300 import binding as F  # noqa: E402


class Model:
    """A pre-norm transformer of random weights over a paged cache: grouped heads, normalised queries and keys."""

    def __init__(self, seed, B, context, vocab, layers, width=256, heads=8, kv_heads=2, head_dim=64, page=16,
                 max_nodes=64, embedding=None, device="cuda", bits=16):
        g = torch.Generator(device=device).manual_seed(seed)

        def mat(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.embedding = mat(vocab, width) * width ** 0.5 if embedding is None else embedding
        self.blocks = [dict(qkv=mat((heads + 2 * kv_heads) * head_dim, width), out=mat(width, heads * head_dim),
                            up=mat(4 * width, width), down=mat(width, 4 * width),
                            qw=torch.ones(head_dim, device=device).bfloat16() * 2,
                            kw=torch.ones(head_dim, device=device).bfloat16()) for _ in range(layers)]
        pages = -(-context // page)
        lengths = torch.zeros(B, dtype=torch.int32, device=device)
        if bits == 4:
            self.pool = F.PagePool(B * pages, page, B, pages, device=device)
            self.cache = F.KVCache4.zeros(layers, B * pages, page, kv_heads, head_dim, self.pool.page_table, lengths)
            self.append, self.attend, self.commit = F.spec_tree_kv4_append, F.spec_tree_kv4_attend, F.spec_tree_kv4_commit
        else:
            self.pool = None
            shape = (layers, B * pages, page, kv_heads, head_dim)
            # without a pool, each sequence owns a shuffled set of pages from the start
            table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(seed)).int().view(B, pages)
            self.cache = F.KVCache(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                                   torch.zeros(shape, dtype=torch.bfloat16, device=device), table.to(device), lengths)
            self.append, self.attend, self.commit = F.spec_tree_kv_append, F.spec_tree_attend, F.spec_tree_kv_commit
        self.rope = F.rope_table(context, head_dim, 10000.0, device)
        self.workspace = F.AttendWorkspace(B, max_nodes, heads, kv_heads, head_dim, device)

    def step(self, tokens, status, tree=None, begin=0):
        """Logits [B][N][vocab] of nodes begin .. begin + N - 1, whose entries are appended to the cache."""
        B, N = tokens.shape
        if self.pool:
            F.spec_tree_kv_reserve(self.pool, self.cache.seq_len, begin + N, status)
        x = self.embedding[tokens.clamp_min(0).long()].float()
        norm = lambda y: (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).bfloat16()  # noqa: E731
        for layer, w in enumerate(self.blocks):
            qkv = (norm(x) @ w["qkv"].T).view(B, N, self.heads + 2 * self.kv_heads, self.head_dim)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=2)
            self.append(self.cache, layer, q, k, v, q, self.rope, status, tree=tree, node_begin=begin, q_weight=w["qw"],
                        k_weight=w["kw"])
            out = torch.empty((B, N, self.heads, self.head_dim), dtype=q.dtype, device=q.device)
            self.attend(self.cache, layer, q, out, self.workspace, status, tree=tree, node_begin=begin)
            x = x + (out.view(B, N, -1) @ w["out"].T).float()
            x = x + (torch.nn.functional.silu(norm(x) @ w["up"].T) @ w["down"].T).float()
        return norm(x) @ self.embedding.T * self.embedding.shape[1] ** -0.5

    def keep(self, lengths, status):
        """The cache's lengths from now on; pages behind them go back to the pool."""
        self.cache.set_lengths(lengths)
        if self.pool:
            F.spec_tree_kv_release(self.pool, lengths, status)


def decode(B=4, rounds=12, vocab=4096, prompt_len=40, seed=0, K=4, W=4, depth=4, R=20, layers=2, bits=16):
    """(target, tokens, accepted): the target model, each sequence's tokens (the last one is not cached yet) and
    the accept lengths of every round."""
    params = F.Params(K=K, m=1, W=W, depth=depth, R=R, temperature=1.0, support=64)
    context = prompt_len + rounds * (depth + 1) + R + 1
    max_nodes = max(R + 1, 1 + (depth - 1) * W, prompt_len)
    target = Model(seed, B, context, vocab, layers, max_nodes=max_nodes, bits=bits)
    drafter = Model(seed + 1, B, context, vocab, 1, max_nodes=max_nodes, embedding=target.embedding, bits=bits)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed + 2)
    uniform = lambda *shape: torch.rand(shape, generator=g, device=dev)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    tree, state, out = F.TreeBuffers(params, B), F.LayerState(params, B), F.VerifyOutputs(params, B)
    new_len = torch.zeros(B, dtype=torch.int32, device=dev)

    # the prompt, a chain; its last token is the first root
    prompt = torch.randint(0, vocab, (B, prompt_len), generator=g, device=dev)
    for model in (target, drafter):
        model.step(prompt[:, :-1], status)
    lengths = torch.full((B,), prompt_len - 1, dtype=torch.int32, device=dev)
    root = prompt[:, -1].int()
    tokens, accepted = [row.tolist() for row in prompt], []

    for _ in range(rounds):
        target.keep(lengths, status)
        drafter.keep(lengths, status)
        # drafting: nodes in the order they are expanded, layer l's at 1 + (l - 1) W
        nodes = 1 + (depth - 1) * W
        parent = torch.full((B, nodes), -1, dtype=torch.int32, device=dev)
        deep = torch.zeros((B, nodes), dtype=torch.int32, device=dev)
        frontier = root[:, None]
        for layer in range(depth):
            rows = F.spec_tree_layer_rows(params, layer)
            begin = 0 if layer == 0 else 1 + (layer - 1) * W
            if layer > 0:
                frontier = state.frontier_token[:, :rows]
                above = 0 if layer == 1 else begin - W + state.frontier_parent[:, :rows]
                parent[:, begin:begin + rows] = above
                deep[:, begin:begin + rows] = layer
            logits = drafter.step(frontier, status, F.NodeArrays(parent, deep), begin)
            F.spec_tree_layer(params, vocab, layer, logits.contiguous(), uniform(B, rows), tree, state, status)
        F.spec_tree_finish(params, vocab, tree, state, status)
        # verification
        ids = tree.node_token.clone()
        ids[:, 0] = root
        logits = target.step(ids, status, tree)
        F.spec_tree_verify(params, vocab, logits.contiguous(), tree, uniform(B, depth, K), uniform(B), out.accept_len,
                           out.out_tok, out.out_node, out.margins, status)
        # commit: the target's entries are moved, the drafter makes its own from the accepted tokens
        target.commit(target.cache, out.accept_len, out.out_node, new_len, status)
        chain = torch.cat([root[:, None], out.out_tok[:, :depth]], 1)
        drafter.step(chain, status, F.NodeArrays(n_nodes=out.accept_len + 1))
        lengths, new_len = new_len, lengths
        root = out.out_tok.gather(1, out.accept_len[:, None].long())[:, 0].contiguous()
        for b, (n, row) in enumerate(zip(out.accept_len.tolist(), out.out_tok.tolist())):
            tokens[b] += row[:n + 1]
        accepted.append(out.accept_len.tolist())
    target.keep(lengths, status)
    torch.cuda.synchronize()
    if int(status.item()):
        raise RuntimeError(f"status {int(status.item())}")
    return target, tokens, accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=12)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--bits", type=int, default=16, choices=(16, 4), help="of the caches' keys and values")
    args = ap.parse_args()
    _, tokens, accepted = decode(B=args.batch, rounds=args.rounds, bits=args.bits)
    total = sum(map(sum, accepted))
    print(f"{args.batch} sequences, {args.rounds} target passes: {total / args.batch / args.rounds:.2f} tokens accepted "
          f"per tree, {len(tokens[0])} tokens in the first sequence")


if __name__ == "__main__":
    main()
