#!/usr/bin/env python3
"""Text from a small quantized decoder, several tokens per pass.

A decoder of seeded Q4_K / Q6_K weights: its linears are rq_linear and
rq_linear_group, its attention runs over a paged 8-bit cache, and its tokens
are drafted from the text so far and verified by the decoder:

  cache slots, positions and pages of the new tokens
          rq_batch_plan
  residual sums and norms between the blocks
          rq_residual_norm
  q/k/v   rq_linear_group     (one launch for the three)
  norm of q and k per head, rotation, quantized write of k and v
          rq_qkv_to_cache     (one pass)
  attention of the last token and its drafts, causal or a tree
          Context.rq_cache_attention
  o, gate/up, down, vocabulary
          rq_linear, rq_linear_group; the gate product of a long prompt
          rq_linear_epilogue
  temperature, top-k, top-p and min-p
          rq_token_probs
  which drafts stay, and the next token
          rq_verify_chain or rq_verify_tree
  accepted tokens of a tree to the places that follow the text
          rq_kv_read, rq_kv_write

    python examples/speculative_decode.py [--drafts none|chain|tree] [--tokens N] [--top-p P]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_layers_gb300 as rq  # noqa: E402
import synthetic  # noqa: E402

Q4K, Q6K = rq.RQ_Q4K, rq.RQ_Q6K


def _weight(seed, qtype, N, K):
    w = np.ascontiguousarray(synthetic.weight_matrix(seed, qtype, N, K))
    return torch.from_numpy(w.view(np.uint8).reshape(-1)).cuda()


def _normal(seed, *shape):
    n = int(np.prod(shape))
    return torch.from_numpy(synthetic.normal_f32(seed, n)[:n].reshape(shape).copy()).cuda()


class Decoder:
    """One sequence through a decoder of `layers` layers and a paged cache."""

    def __init__(self, layers=2, hidden=1024, heads=8, kv_heads=2, head_dim=128,
                 intermediate=2048, vocab=512, page_size=16, max_tokens=512,
                 format=rq.RQ_KV_E4M3, seed=1):
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.intermediate, self.vocab, self.max_tokens = intermediate, vocab, max_tokens
        # Below the threshold a token's linears are the same sums however many
        # tokens a pass has, so that drafts do not change the text.
        self.ctx = rq.Context(gemm_threshold=65)
        d, q, kv = head_dim, heads * head_dim, kv_heads * head_dim
        self.embedding = _normal(synthetic.substream(seed, 0), vocab, hidden)
        self.head = _weight(synthetic.substream(seed, 1), Q6K, vocab, hidden)
        angle = torch.arange(max_tokens).double()[:, None] * 10000.0 ** (
            -torch.arange(0, d, 2).double() / d)
        cos, sin = angle.cos().float().cuda(), angle.sin().float().cuda()
        self.layers = []
        # unused pages in an order of their own: a page is found by the table only
        pages = (max_tokens + page_size - 1) // page_size
        self.free = torch.from_numpy(
            np.argsort(synthetic.u64(synthetic.substream(seed, 2), pages)).astype(np.int32)).cuda()
        self.left = torch.empty(1, dtype=torch.int32, device="cuda")
        self.table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
        self.slot = None
        # a norm after each block and before the next, without weights of their own
        self.first_norm = rq.NormParams(hidden, post=False)
        self.norms = rq.NormParams(hidden)
        for i in range(layers):
            s = [synthetic.substream(seed, 100 * (i + 1) + j) for j in range(9)]
            self.layers.append(dict(
                types=[Q4K, Q4K, Q6K], rows=[q, kv, kv],
                qkv=[_weight(s[0], Q4K, q, hidden), _weight(s[1], Q4K, kv, hidden),
                     _weight(s[2], Q6K, kv, hidden)],
                o=_weight(s[3], Q4K, hidden, q),
                up=[_weight(s[4], Q4K, intermediate, hidden),
                    _weight(s[5], Q4K, intermediate, hidden)],
                down=_weight(s[6], Q4K, hidden, intermediate),
                params=rq.QKParams(heads, kv_heads, d, 1.0 + 0.1 * _normal(s[7], d),
                                   1.0 + 0.1 * _normal(s[8], d), 1e-6, cos, sin),
                cache=rq.KVCache(pages, page_size, kv_heads, d, format)))
        self.page_size = page_size

    def forward(self, tokens, length, depth=None, tree=None):
        """Logits [n, vocab] after each of n new tokens that follow `length`
        cached ones; depth: their places in the text beyond length, and tree
        the new tokens that each sees (None: one after another)."""
        n = len(tokens)
        assert length + n <= self.max_tokens
        lengths = torch.tensor([length], dtype=torch.int32, device="cuda")
        # the first pages of the stack's end hold the text; those that drafts
        # took which were not kept are taken again
        held = -(-length // self.page_size)
        count = torch.tensor([len(self.free) - held], dtype=torch.int32, device="cuda")
        slot = self.slot = torch.empty(n, dtype=torch.int64, device="cuda")
        position = torch.empty(n, dtype=torch.int32, device="cuda")
        rq.rq_batch_plan(lengths, self.table, self.free, count, self.left, slot, position,
                         self.page_size, new_tokens=n)
        if depth is not None:
            position = (length + torch.tensor(depth, device="cuda")).int()
        words = None
        if tree is not None:
            words = torch.tensor([tree], dtype=torch.int64, device="cuda")

        def f32(cols):
            return torch.empty(n, cols, device="cuda")

        x = self.embedding[torch.tensor(tokens, device="cuda")]
        normed = f32(self.hidden)
        rq.rq_residual_norm(self.first_norm, None, x, None, normed, n)
        for layer in self.layers:
            qkv = [f32(rows) for rows in layer["rows"]]
            self.ctx.rq_act_cache_invalidate()      # normed is written in place
            self.ctx.rq_linear_group(layer["types"], layer["qkv"], normed, qkv, layer["rows"], n,
                                     self.hidden)
            q, k, v = (t.view(n, -1, self.head_dim) for t in qkv)
            rq.rq_qkv_to_cache(layer["params"], q, k, v, position, q, layer["cache"], slot, n)
            out = torch.empty_like(q)
            self.ctx.rq_cache_attention(layer["cache"], q, out, self.table, lengths, 1, n,
                                        self.heads, self.head_dim ** -0.5, tree=words)
            y = f32(self.hidden)
            self.ctx.rq_linear(Q4K, layer["o"], out, y, n, self.hidden,
                               self.heads * self.head_dim)
            rq.rq_residual_norm(self.norms, y, x, x, normed, n)
            self.ctx.rq_act_cache_invalidate()
            gate, up = f32(self.intermediate), f32(self.intermediate)
            if n < self.ctx.gemm_threshold:
                self.ctx.rq_linear_group([Q4K, Q4K], layer["up"], normed, [gate, up],
                                         [self.intermediate] * 2, n, self.hidden)
                gated = torch.nn.functional.silu(gate) * up
            else:
                self.ctx.rq_linear(Q4K, layer["up"][1], normed, up, n, self.intermediate,
                                   self.hidden)
                self.ctx.rq_linear_epilogue(Q4K, layer["up"][0], normed, gate, n,
                                            self.intermediate, self.hidden, act="silu", mul=up)
                gated = gate
            self.ctx.rq_linear(Q4K, layer["down"], gated, y, n, self.hidden, self.intermediate)
            rq.rq_residual_norm(self.norms, y, x, x, normed, n)
        self.ctx.rq_act_cache_invalidate()
        logits = f32(self.vocab)
        self.ctx.rq_linear(Q6K, self.head, normed, logits, n, self.vocab, self.hidden)
        return logits

    def keep(self, length, path):
        """Moves the accepted tokens of a tree, new tokens path[0] < path[1] <
        ..., to the places that follow `length`."""
        if list(path) == list(range(len(path))):
            return
        n = len(path)
        old = self.slot[torch.tensor(path, device="cuda")]
        new = self.slot[:n].contiguous()
        for layer in self.layers:
            k = torch.empty(n, self.kv_heads, self.head_dim, device="cuda")
            v = torch.empty_like(k)
            rq.rq_kv_read(layer["cache"], old, k, v, n)
            rq.rq_kv_write(layer["cache"], k, v, new, n)


def continuations(text, width, depth):
    """Drafts from the text itself: what followed its last token at the `width`
    latest places where that token stood before, `depth` tokens each."""
    found = []
    for i in range(len(text) - 2, -1, -1):
        if text[i] == text[-1]:
            run = text[i + 1:i + 1 + depth]
            if run not in found:
                found.append(run)
            if len(found) == width:
                break
    return found


def as_tree(runs):
    """(tokens, parents) of the runs with equal beginnings joined."""
    tokens, parents = [], []
    for run in runs:
        at = -1
        for t in run:
            for i, (u, p) in enumerate(zip(tokens, parents)):
                if u == t and p == at:
                    at = i
                    break
            else:
                tokens.append(t)
                parents.append(at)
                at = len(tokens) - 1
    return tokens, parents


def generate(decoder, prompt, count, drafts="tree", width=3, depth=4, temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0, seed=7):
    """(`count` tokens after the prompt, passes that took): with a tree or
    without drafts the draw at each place uses that place's random number, so
    both write the same text."""
    u = synthetic.uniform(seed, decoder.max_tokens + 1).astype(np.float32)
    u = np.minimum(u, np.float32(1.0 - 2.0 ** -24))
    text, passes, length = list(prompt), 0, len(prompt) - 1
    if length > 0:
        decoder.forward(text[:-1], 0)  # the prompt into the cache
    while len(text) < len(prompt) + count:
        runs = [] if drafts == "none" else continuations(text, 1 if drafts == "chain" else width,
                                                         depth)
        tokens, parents = as_tree(runs)
        n = len(tokens)
        new = [text[-1]] + tokens
        levels, sees = [0], [1]
        for i, p in enumerate(parents):
            levels.append(levels[p + 1] + 1)
            sees.append(sees[p + 1] | 1 << (i + 1))
        logits = decoder.forward(new, length, levels, sees if drafts == "tree" else None)
        passes += 1
        rows = len(new)
        p = torch.empty(1, rows, decoder.vocab, device="cuda")
        rq.rq_token_probs(logits, p, rows, decoder.vocab,
                          temperature=torch.full((rows,), temperature, device="cuda"),
                          top_k=torch.full((rows,), top_k, dtype=torch.int32, device="cuda"),
                          top_p=torch.full((rows,), top_p, device="cuda"),
                          min_p=torch.full((rows,), min_p, device="cuda"))
        token = torch.tensor([tokens], dtype=torch.int32, device="cuda")
        accepted = torch.empty(1, dtype=torch.int32, device="cuda")
        following = torch.empty_like(accepted)
        # the number that decides what stands at a place of the text
        random = torch.from_numpy(u[[length + 1 + level for level in levels]])[None].cuda()
        if drafts == "chain":
            rq.rq_verify_chain(token, p, None, random, accepted, following, 1, n, decoder.vocab)
            path = list(range(int(accepted)))
        else:
            parent = torch.tensor([parents], dtype=torch.int32, device="cuda")
            walked = torch.empty(1, max(n, 1), dtype=torch.int32, device="cuda")
            rq.rq_verify_tree(token, parent, p, random, accepted, following, walked, 1, n,
                              decoder.vocab)
            path = walked[0, :int(accepted)].tolist()
        decoder.keep(length, [0] + [i + 1 for i in path])
        text += [tokens[i] for i in path] + [int(following)]
        length += 1 + len(path)
    status = rq.rq_get_device_status()
    if status != 0:
        raise rq.RqError(status, "generate")
    return text[len(prompt):len(prompt) + count], passes


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--drafts", choices=("none", "chain", "tree"), default="tree")
    ap.add_argument("--tokens", type=int, default=96)
    ap.add_argument("--temperature", type=float, default=0.5)
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    args = ap.parse_args()
    text, passes = generate(Decoder(), [3, 141, 59, 26, 53], args.tokens, args.drafts,
                            temperature=args.temperature, top_k=args.top_k, top_p=args.top_p,
                            min_p=args.min_p)
    print(" ".join(map(str, text)))
    print("%d tokens in %d passes" % (len(text), passes))


if __name__ == "__main__":
    main()
