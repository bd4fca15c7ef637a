"""Shared parts of the cache, attention and verification tests: plain 64-bit
definitions on the CPU."""
import math

import numpy as np
import torch

TOP = {0: 448.0, 1: 127.0}          # RQ_KV_E4M3, RQ_KV_I8
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # unit roundoff
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def encode(x, fmt):
    """Codes and scales of f32 rows by the cache's definition (CPU, f32)."""
    top = torch.tensor(TOP[fmt])
    fin = torch.isfinite(x)
    a = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(-1, keepdim=True)
    a = a.clamp_min(2.0 ** -100)
    y = torch.where(fin, x * (top * (torch.tensor(1.0) / a)), torch.copysign(top, x)).clamp(-top, top)
    codes = y.to(torch.float8_e4m3fn) if fmt == 0 else y.round().to(torch.int8)
    return codes, (a / top).squeeze(-1)


def random_pool(seed, pages, hk, page, d, fmt):
    """Codes and scales of normal rows, on the CPU."""
    g = gen(seed)
    k, ks = encode(torch.randn((pages, hk, page, d), generator=g), fmt)
    v, vs = encode(torch.randn((pages, hk, page, d), generator=g), fmt)
    return k, v, ks, vs


def values(codes, scales):
    return codes.float().double() * scales.double()[..., None]


def attention(q, k, v, table, lengths, tree, scale, fmt_dtype, page):
    """The definition in 64 bits, and its error bound per output.

    q [b, new, h, d] (CPU), k / v dequantized pools [pages, hk, page, d] in 64
    bits.  The bound: scores carry q's split and the f32 sums of d products,
    the probabilities twice the largest score error and their f16 rounding
    (22 bits with f32 activations), the output its own f32 sums and the last
    rounding."""
    b, new, h, d = q.shape
    hk = k.shape[1]
    out = torch.zeros((b, new, h, d), dtype=torch.float64)
    tol = torch.zeros_like(out)
    q = q.double()
    for i in range(b):
        n = int(lengths[i])
        if n < 0:
            continue
        total = n + new
        pages = table[i, :-(-total // page)].long()
        kk = k[pages].permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :total]
        vv = v[pages].permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :total]
        open_ = torch.zeros((new, total), dtype=torch.bool)
        open_[:, :n] = True
        for r in range(new):
            for c in range(new):
                if tree is None:
                    open_[r, n + c] = c <= r
                else:
                    open_[r, n + c] = bool((int(tree[i, r]) >> c) & 1)
        for head in range(h):
            kh, vh = kk[head // (h // hk)], vv[head // (h // hk)]
            # what is masked may hold anything: it is cut out, not multiplied by 0
            for r in range(new):
                sel = open_[r]
                if not bool(sel.any()):
                    continue
                ks, vs = kh[sel], vh[sel]
                s = scale * (ks @ q[i, r, head])
                p = torch.softmax(s, 0)
                out[i, r, head] = p @ vs
                size = float((scale * (ks.abs() @ q[i, r, head].abs())).max())
                ds = (2.0 ** -22 + (d / 16 + 16) * 2.0 ** -23) * size
                pr = 2.0 ** -21 if fmt_dtype == "f32" else 2.0 ** -11
                rel = 2 * ds + pr + (total / 64 + 64) * 2.0 ** -22
                tol[i, r, head] = rel * (p @ vs.abs()) + 2.0 ** -30 * float(vs.abs().max())
    tol += ROUND[fmt_dtype] * out.abs() * 1.01 + (2.0 ** -25 if fmt_dtype == "f16" else 0.0)
    return out, tol


def draw(w, u):
    """The integer draw: token index, or -1 (w: f32 numpy row)."""
    w = np.where(w > 0, np.minimum(w, np.float32(1)), np.float32(0)).astype(np.float64)
    W = [int(x) for x in np.floor(w * 2.0 ** 36)]
    total = sum(W)
    if total == 0:
        return -1
    un = min(max(int(math.floor(float(u) * 2.0 ** 24)), 0), (1 << 24) - 1) if u == u else 0
    point, run = un * total >> 24, 0
    for i, x in enumerate(W):
        run += x
        if run > point:
            return i
    raise AssertionError


def verify_chain(tok, p, q, u):
    n = len(tok)
    V = p.shape[1]
    for i in range(n):
        x = int(tok[i])
        if not 0 <= x < V:
            return i, draw(p[i], u[n])
        t = u[i] * q[i, x] if q is not None else u[i]
        if not t < p[i, x]:
            w = p[i] - q[i] if q is not None else p[i].copy()
            if q is None:
                w[x] = 0
            y = draw(w, u[n])
            return i, y if y >= 0 else draw(p[i], u[n])
    return n, draw(p[n], u[n])


def verify_tree(tok, par, p, u):
    node, path = -1, []
    while True:
        y = draw(p[node + 1], u[node + 1])
        nxt = [i for i in range(len(tok)) if par[i] == node and tok[i] == y and par[i] < i]
        if y < 0 or not nxt:
            return path, y
        node = nxt[0]
        path.append(node)
