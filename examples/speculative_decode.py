#!/usr/bin/env python3
"""Text from a small quantized decoder, several tokens per pass.

A decoder of seeded Q4_K / Q6_K weights: its linears are rq_linear and
rq_linear_group, its attention runs over a paged 8-bit cache, and its tokens
are drafted from the text so far and verified by the decoder:

  q/k/v   rq_linear_group     (one launch for the three)
  norm of q and k per head, rotation, quantized write of k and v
          rq_qkv_to_cache     (one pass)
  attention of the last token and its drafts, causal or a tree
          Context.rq_cache_attention
  o, gate/up, down, vocabulary
          rq_linear, rq_linear_group
  which drafts stay, and the next token
          rq_verify_chain or rq_verify_tree
  accepted tokens of a tree to the places that follow the text
          rq_kv_read, rq_kv_write

    python examples/speculative_decode.py [--drafts none|chain|tree] [--tokens N]
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


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


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
        # pages in an order of their own: a page is found by the table only
        pages = (max_tokens + page_size - 1) // page_size
        self.table = torch.from_numpy(
            np.argsort(synthetic.u64(synthetic.substream(seed, 2), pages)).astype(np.int32)).cuda()
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

    def slots(self, places):
        """Cache slots of places in the text (int64 tensor on the device)."""
        page = self.table[places // self.page_size].long()
        return page * self.page_size + places % self.page_size

    def forward(self, tokens, length, depth=None, tree=None):
        """Logits [n, vocab] after each of n new tokens that follow `length`
        cached ones; depth: their places in the text beyond length, and tree
        the new tokens that each sees (None: one after another)."""
        n = len(tokens)
        assert length + n <= self.max_tokens
        place = length + torch.arange(n, device="cuda")
        slot = self.slots(place)
        position = (place if depth is None else
                    length + torch.tensor(depth, device="cuda")).int()
        lengths = torch.tensor([length], dtype=torch.int32, device="cuda")
        words = None
        if tree is not None:
            words = torch.tensor([tree], dtype=torch.int64, device="cuda")

        def f32(cols):
            return torch.empty(n, cols, device="cuda")

        x = self.embedding[torch.tensor(tokens, device="cuda")]
        for layer in self.layers:
            qkv = [f32(rows) for rows in layer["rows"]]
            self.ctx.rq_linear_group(layer["types"], layer["qkv"], _rms(x), qkv, layer["rows"], n,
                                     self.hidden)
            q, k, v = (t.view(n, -1, self.head_dim) for t in qkv)
            rq.rq_qkv_to_cache(layer["params"], q, k, v, position, q, layer["cache"], slot, n)
            out = torch.empty_like(q)
            self.ctx.rq_cache_attention(layer["cache"], q, out, self.table[None], lengths, 1, n,
                                        self.heads, self.head_dim ** -0.5, tree=words)
            y = f32(self.hidden)
            self.ctx.rq_linear(Q4K, layer["o"], out, y, n, self.hidden,
                               self.heads * self.head_dim)
            x = x + _rms(y)
            gate, up = f32(self.intermediate), f32(self.intermediate)
            self.ctx.rq_linear_group([Q4K, Q4K], layer["up"], _rms(x), [gate, up],
                                     [self.intermediate] * 2, n, self.hidden)
            y = f32(self.hidden)
            self.ctx.rq_linear(Q4K, layer["down"], torch.nn.functional.silu(gate) * up, y, n,
                               self.hidden, self.intermediate)
            x = x + _rms(y)
        logits = f32(self.vocab)
        self.ctx.rq_linear(Q6K, self.head, _rms(x), logits, n, self.vocab, self.hidden)
        return logits

    def keep(self, length, path):
        """Moves the accepted tokens of a tree, new tokens path[0] < path[1] <
        ..., to the places that follow `length`."""
        if list(path) == list(range(len(path))):
            return
        n = len(path)
        old = self.slots(length + torch.tensor(path, device="cuda"))
        new = self.slots(length + torch.arange(n, device="cuda"))
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


def generate(decoder, prompt, count, drafts="tree", width=3, depth=4, temperature=1.0, seed=7):
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
        p = torch.softmax(logits / temperature, -1)[None]
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
    args = ap.parse_args()
    text, passes = generate(Decoder(), [3, 141, 59, 26, 53], args.tokens, args.drafts,
                            temperature=args.temperature)
    print(" ".join(map(str, text)))
    print("%d tokens in %d passes" % (len(text), passes))


if __name__ == "__main__":
    main()
