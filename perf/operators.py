"""The serving operators around the quantized linear layer, as measurable cases.

Four operators carry a decoder layer from its q/k/v products to the next
token: per-head norms and position rotation of q and k with the quantized
cache write in the same pass ("qkv"), the quantized cache's write and read
back ("kv_write", "kv_read"), attention of single tokens, drafted trees and
prompts over the paged quantized cache ("attention"), and the verification of
drafted tokens against the target's probabilities ("verify").

With `own` false, run() computes a case with elementary torch operations in
32 bits; with `own` true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2}
TOP = {"e4m3": 448.0, "i8": 127.0}
TINY = 2.0 ** -100          # least maximum a scale is taken from
EPS = 1e-6


def _rq():
    import quantized_linear_layers_gb300 as rq
    return rq


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step's q, k, v of one sequence, as rq_linear_group leaves
        # them (28 / 4 heads of 128): latency counts
        dict(name="qkv_one_token", op="qkv", tokens=1, q_heads=28, kv_heads=4, head_dim=128,
             rotary=128, interleaved=False, packed=False, dtype="f32", format="e4m3", page=64),
        # a batch of drafted tokens cut out of one packed q|k|v buffer, half of
        # each head rotated, pairs side by side, 8-bit integer cache
        dict(name="qkv_drafts", op="qkv", tokens=200, q_heads=32, kv_heads=8, head_dim=128,
             rotary=64, interleaved=True, packed=True, dtype="bf16", format="i8", page=16),
        # a prompt of the decoder's longest prefill
        dict(name="qkv_prompt", op="qkv", tokens=4096, q_heads=28, kv_heads=4, head_dim=128,
             rotary=128, interleaved=False, packed=False, dtype="f32", format="e4m3", page=64),
        # keys and values that need no rotation (an imported prefix), narrow heads
        dict(name="kv_write_1500", op="kv_write", tokens=1500, kv_heads=8, head_dim=64,
             dtype="f16", format="i8", page=32),
        # a long prefix read back to hand it to another program
        dict(name="kv_read_30000", op="kv_read", tokens=30000, kv_heads=4, head_dim=128,
             dtype="bf16", format="e4m3", page=64),
        # one token of a chat just begun
        dict(name="attn_one_short", op="attention", batch=1, new=1, context=500, tree=False,
             q_heads=28, kv_heads=4, head_dim=128, dtype="f32", format="e4m3", page=64),
        # one token at the end of a very long document
        dict(name="attn_one_long", op="attention", batch=1, new=1, context=131000, tree=False,
             q_heads=28, kv_heads=4, head_dim=128, dtype="f32", format="e4m3", page=64),
        # a serving batch, one token each, lengths from half the longest on
        dict(name="attn_batch", op="attention", batch=64, new=1, context=8192, tree=False,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", format="i8", page=16),
        # drafted trees over a cache, a handful of sequences
        dict(name="attn_tree", op="attention", batch=8, new=48, context=8000, tree=True,
             q_heads=28, kv_heads=4, head_dim=128, dtype="f32", format="e4m3", page=64),
        # the rest of two prompts behind a shared prefix
        dict(name="attn_prompt", op="attention", batch=2, new=1500, context=600, tree=False,
             q_heads=28, kv_heads=4, head_dim=128, dtype="bf16", format="e4m3", page=128),
        # chains of seven drafts with their draft distributions
        dict(name="verify_chain", op="verify", batch=32, drafts=7, vocab=131072, tree=False),
        # trees of forty drafts, odd vocabulary
        dict(name="verify_tree", op="verify", batch=6, drafts=40, vocab=50001, tree=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["qkv", "qkv", "kv_write", "kv_read", "attention", "attention", "attention",
                     "verify", "verify"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    fmt = rng.choice(["e4m3", "i8"])
    page = rng.choice([16, 32, 64, 128])
    q_heads, kv_heads, head_dim = rng.choice(
        [(28, 4, 128), (32, 8, 128), (16, 16, 128), (10, 2, 64), (14, 2, 64), (8, 1, 256),
         (5, 5, 64), (40, 8, 128)])
    heads = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim)
    if op == "qkv":
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        return dict(op=op, tokens=_log(rng, 1, 2500), **heads, rotary=rotary,
                    interleaved=rng.random() < 0.4, packed=rng.random() < 0.5, dtype=dtype,
                    format=fmt, page=page)
    if op in ("kv_write", "kv_read"):
        return dict(op=op, tokens=_log(rng, 1, 20000), kv_heads=kv_heads, head_dim=head_dim,
                    dtype=dtype, format=fmt, page=page)
    if op == "attention":
        kind = rng.choice(["one", "one", "tree", "prompt"])
        if kind == "one":
            batch = _log(rng, 1, 64)
            new, context = 1, _log(rng, 1, min(60000, 260000 // batch))
        elif kind == "tree":
            batch = _log(rng, 1, 16)
            new, context = rng.randint(2, 64), _log(rng, 1, min(20000, 64000 // batch))
        else:
            batch = rng.randint(1, 3)
            new, context = _log(rng, 65, 1000), _log(rng, 1, 1000)
        return dict(op=op, batch=batch, new=new, context=context, tree=kind == "tree", **heads,
                    dtype=dtype, format=fmt, page=page)
    tree = rng.random() < 0.5
    return dict(op=op, batch=_log(rng, 1, 32 if not tree else 8),
                drafts=rng.randint(1, 12 if not tree else 64), vocab=_log(rng, 1000, 100000),
                tree=tree)


def _lengths(case):
    """Cached tokens of each sequence before the new ones: the case's context,
    or for a batch spread evenly from half of it on."""
    b, c = case["batch"], case["context"]
    return [c - (c // 2) * ((7 * i) % b) // b for i in range(b)]


def _parents(case):
    """Three drafts after the last token, three after each of the first drafts
    and so on, in order of depth: -1 is the last token itself."""
    n = case["new"] if case["op"] == "attention" else case["drafts"]
    return [i // 3 - 1 for i in range(n)]


def work(case):
    op = case["op"]
    if op == "qkv":
        t, d = case["tokens"], case["head_dim"]
        q, kv, w = t * case["q_heads"] * d, t * case["kv_heads"] * d, WIDTH[case["dtype"]]
        read = (q + 2 * kv) * w + t * (case["rotary"] * 4 + 4 + 8)
        wrote = q * w + 2 * kv + 2 * t * case["kv_heads"] * 4
        if case["format"] == "i8":      # read back in 16 bits
            wrote += 2 * kv * 2
        return {"bytes": read + wrote, "flops": 8 * q + 12 * kv}
    if op in ("kv_write", "kv_read"):
        rows = case["tokens"] * case["kv_heads"]
        n = rows * case["head_dim"]
        return {"bytes": 2 * n * (WIDTH[case["dtype"]] + 1) + 8 * rows + 8 * case["tokens"],
                "flops": 4 * n}
    if op == "attention":
        d, h, new = case["head_dim"], case["q_heads"], case["new"]
        q = case["batch"] * new * h * d
        cached = sum(n + new for n in _lengths(case)) * case["kv_heads"]
        if case["tree"]:
            depth, seen = [], 0
            for p in _parents(case):
                depth.append(1 if p < 0 else depth[p] + 1)
            seen = sum(n * new + sum(depth) for n in _lengths(case))
        else:
            seen = sum(n * new + new * (new + 1) // 2 for n in _lengths(case))
        return {"bytes": cached * 2 * (d + 4) + 2 * q * WIDTH[case["dtype"]],
                "flops": 4 * seen * h * d}
    b, v = case["batch"], case["vocab"]
    # the one row that the next token is drawn from (and its draft's), or in a
    # tree the last token's row at least
    rows = 1 if case["tree"] else 2
    return {"bytes": b * rows * v * 4, "flops": b * rows * v * 2}


# ----------------------------------------------------------------- inputs --

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _activations(g, shape, dtype, device):
    """N(0, 1) with one entry in a thousand 20 times larger."""
    x = torch.randn(shape, generator=g, device=device)
    x = torch.where(torch.rand(shape, generator=g, device=device) < 1e-3, 20.0 * x, x)
    return x.to(DTYPES[dtype])


def _encode(x, fmt):
    """Codes and scales of rows (last axis) of 32-bit x: scale = A / top with
    A the row's largest finite magnitude, code = x * (top / A) rounded to even;
    what is not finite takes its sign's largest code."""
    top = TOP[fmt]
    finite = torch.isfinite(x)
    a = torch.where(finite, x.abs(), torch.zeros_like(x)).amax(-1, keepdim=True).clamp_min(TINY)
    y = (x * (top / a)).clamp(-top, top)
    y = torch.where(finite, y, torch.copysign(torch.full_like(x, top), x))
    codes = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(y).to(torch.int8)
    return codes, (a / top).squeeze(-1)


def _pool(case, pages, device):
    shape = (pages, case["kv_heads"], case["page"])
    code = torch.float8_e4m3fn if case["format"] == "e4m3" else torch.int8
    return dict(k=torch.zeros(shape + (case["head_dim"],), dtype=torch.uint8, device=device).view(code),
                v=torch.zeros(shape + (case["head_dim"],), dtype=torch.uint8, device=device).view(code),
                ks=torch.zeros(shape, device=device), vs=torch.zeros(shape, device=device))


def _handle(case, s):
    """The framework's description of the cache, kept as a user's program keeps it."""
    rq = _rq()
    fmt = rq.RQ_KV_E4M3 if case["format"] == "e4m3" else rq.RQ_KV_I8
    s["cache"] = rq.KVCache.from_tensors(s["k"], s["v"], s["ks"], s["vs"], format=fmt)


def _prepare_rows(case, seed, device):
    g = _gen(seed, device)
    t, d, hk = case["tokens"], case["head_dim"], case["kv_heads"]
    page = case["page"]
    pages = -(-t // page) + 3
    s = dict(case=case, **_pool(case, pages, device))
    # the tokens' places: pages handed out in no order
    order = torch.randperm(pages, generator=g, device=device)
    at = torch.arange(t, device=device)
    s["slots"] = order[at // page] * page + at % page
    if case["op"] == "kv_read":
        for c, sc in (("k", "ks"), ("v", "vs")):
            codes, scale = _encode(torch.randn(s[c].shape, generator=g, device=device), case["format"])
            s[c].view(torch.uint8).copy_(codes.view(torch.uint8))
            s[sc].copy_(scale)
        s["k_out"] = torch.empty((t, hk, d), dtype=DTYPES[case["dtype"]], device=device)
        s["v_out"] = torch.empty_like(s["k_out"])
    elif case["op"] == "kv_write":
        s["k_in"] = _activations(g, (t, hk, d), case["dtype"], device)
        s["v_in"] = _activations(g, (t, hk, d), case["dtype"], device)
    else:
        h, r = case["q_heads"], case["rotary"]
        if case["packed"]:
            x = _activations(g, (t, h + 2 * hk, d), case["dtype"], device)
            s["q_in"], s["k_in"], s["v_in"] = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        else:
            s["q_in"] = _activations(g, (t, h, d), case["dtype"], device)
            s["k_in"] = _activations(g, (t, hk, d), case["dtype"], device)
            s["v_in"] = _activations(g, (t, hk, d), case["dtype"], device)
        s["qw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=device)
        s["kw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=device)
        most = 8192
        angle = torch.arange(most, dtype=torch.float64, device=device)[:, None] * torch.pow(
            torch.tensor(10000.0, dtype=torch.float64, device=device),
            -torch.arange(r // 2, dtype=torch.float64, device=device) * 2 / r)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = int(torch.randint(0, most - t, (1,), generator=g, device=device))
        s["positions"] = (start + at).to(torch.int32)
        s["q_out"] = torch.empty((t, h, d), dtype=DTYPES[case["dtype"]], device=device)
        s["k_back"] = torch.empty((t, hk, d), dtype=torch.bfloat16, device=device)
        s["v_back"] = torch.empty((t, hk, d), dtype=torch.bfloat16, device=device)
        if own:
            s["layer"] = _rq().QKParams(h, hk, d, q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                        cos=s["cos"], sin=s["sin"], rotary_dim=r,
                                        interleaved=case["interleaved"])
    if own:
        _handle(case, s)
    return s


def _tree_bits(parents):
    """Bit j of word i: draft j is draft i or before it on its path."""
    words = []
    for i, p in enumerate(parents):
        words.append((1 << i) | (words[p] if p >= 0 else 0))
    return [w - (1 << 64) if w >> 63 else w for w in words]


def _prepare_attention(case, seed, device):
    g = _gen(seed, device)
    b, new, d = case["batch"], case["new"], case["head_dim"]
    page, hk, h = case["page"], case["kv_heads"], case["q_heads"]
    lengths = _lengths(case)
    most = -(-(max(lengths) + new) // page)
    need = [-(-(n + new) // page) for n in lengths]
    pages = sum(need) + 1
    s = dict(case=case, **_pool(case, pages, device))
    # keys with a few strong channels, as after a norm with learned weights
    channel = 1.0 + 2.0 * (torch.rand(d, generator=g, device=device) < 0.05)
    for c, sc, ch in (("k", "ks", channel), ("v", "vs", torch.ones_like(channel))):
        codes, scale = _encode(torch.randn(s[c].shape, generator=g, device=device) * ch, case["format"])
        s[c].view(torch.uint8).copy_(codes.view(torch.uint8))
        s[sc].copy_(scale)
    order = torch.randperm(pages, generator=g, device=device).to(torch.int32)
    table = torch.zeros((b, most), dtype=torch.int32, device=device)
    first = 0
    for i, n in enumerate(need):
        table[i, :n] = order[first:first + n]
        first += n
    s["table"] = table
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=device)
    s["q"] = torch.randn((b, new, h, d), generator=g, device=device).to(DTYPES[case["dtype"]])
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = d ** -0.5
    s["tree"] = None
    if case["tree"]:
        s["tree"] = torch.tensor(_tree_bits(_parents(case)), dtype=torch.int64,
                                 device=device).repeat(b, 1)
    if own:
        _handle(case, s)
        s["ctx"] = _rq().Context()
    return s


def _prepare_verify(case, seed, device):
    g = _gen(seed, device)
    b, n, v = case["batch"], case["drafts"], case["vocab"]
    s = dict(case=case)
    logits = 2.5 * torch.randn((b, n + 1, v), generator=g, device=device)
    s["u"] = torch.rand((b, n + 1), generator=g, device=device)
    if case["tree"]:
        s["p"] = torch.softmax(logits, -1)
        parents = torch.tensor(_parents(case), device=device)
        # the children of a node: its likeliest tokens, which the node's draw
        # often meets
        best = s["p"].topk(3, dim=-1).indices
        child = torch.arange(n, device=device) % 3
        s["tokens"] = best[:, parents + 1, child].to(torch.int32).contiguous()
        s["parents"] = parents.to(torch.int32).repeat(b, 1)
        # some draws meet the first child, as a good draft's do
        aim = s["p"].gather(-1, best[:, :, :1]).squeeze(-1)
        lower = (s["p"].cumsum(-1).gather(-1, best[:, :, :1]).squeeze(-1) - 0.5 * aim).clamp(0, 0.9999)
        s["u"] = torch.where(torch.rand((b, n + 1), generator=g, device=device) < 0.6, lower, s["u"])
    else:
        s["q"] = torch.softmax(logits[:, :n], -1)
        s["p"] = torch.softmax(
            logits + 0.4 * torch.randn((b, n + 1, v), generator=g, device=device), -1)
        s["tokens"] = torch.multinomial(s["q"].reshape(b * n, v), 1, generator=g).reshape(b, n).to(torch.int32)
    s["accepted"] = torch.empty(b, dtype=torch.int32, device=device)
    s["next"] = torch.empty(b, dtype=torch.int32, device=device)
    s["path"] = torch.empty((b, n), dtype=torch.int32, device=device)
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    if case["op"] == "attention":
        return _prepare_attention(case, seed, device)
    if case["op"] == "verify":
        return _prepare_verify(case, seed, device)
    return _prepare_rows(case, seed, device)


# ------------------------------------------------- the operators in torch --

def _plain_rotate(x, cos, sin, rotary, interleaved):
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = r[..., :rotary // 2], r[..., rotary // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _plain_store(s, k, v):
    case = s["case"]
    page, offset = s["slots"] // case["page"], s["slots"] % case["page"]
    for x, c, sc in ((k, "k", "ks"), (v, "v", "vs")):
        codes, scale = _encode(x, case["format"])
        s[c].view(torch.uint8)[page, :, offset] = codes.view(torch.uint8)
        s[sc][page, :, offset] = scale


def _plain_load(s, slots):
    case = s["case"]
    page, offset = slots // case["page"], slots % case["page"]
    code = s["k"].dtype
    k = s["k"].view(torch.uint8)[page, :, offset].view(code).float() * s["ks"][page, :, offset][..., None]
    v = s["v"].view(torch.uint8)[page, :, offset].view(code).float() * s["vs"][page, :, offset][..., None]
    return k, v


def _plain_rows(s):
    case = s["case"]
    if case["op"] == "kv_read":
        k, v = _plain_load(s, s["slots"])
        return k.to(DTYPES[case["dtype"]]), v.to(DTYPES[case["dtype"]])
    k, v = s["k_in"].float(), s["v_in"].float()
    if case["op"] == "kv_write":
        _plain_store(s, k, v)
        return None
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    turn = (cos, sin, case["rotary"], case["interleaved"])
    q = _plain_rotate(_plain_norm(s["q_in"].float(), s["qw"]), *turn)
    _plain_store(s, _plain_rotate(_plain_norm(k, s["kw"]), *turn), v)
    return q.to(DTYPES[case["dtype"]])


def _plain_attention(s):
    case = s["case"]
    b, new, h, hk, d = (case[n] for n in ("batch", "new", "q_heads", "kv_heads", "head_dim"))
    page = case["page"]
    keys = s["table"].shape[1] * page
    at = torch.arange(keys, device=s["q"].device)
    slots = s["table"].long()[:, at // page] * page + at % page
    k, v = _plain_load(s, slots)                                   # [b, keys, hk, d]
    k, v = k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3)
    q = s["q"].float().view(b, new, hk, h // hk, d).permute(0, 2, 1, 3, 4)
    score = torch.matmul(q.reshape(b, hk, -1, d) * s["scale"], k).view(b, hk, new, h // hk, keys)
    draft = at - s["lengths"].long()[:, None]                      # [b, keys]; negative: cached before
    row = torch.arange(new, device=at.device)
    if s["tree"] is None:
        seen = draft[:, None, :] <= row[:, None]
    else:
        bit = (s["tree"][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
        seen = (draft < 0)[:, None, :] | ((bit == 1) & (draft < new)[:, None, :])
    seen = seen[:, None, :, None, :]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hk, -1, keys), v).view(b, hk, new, h // hk, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.permute(0, 2, 1, 3, 4).reshape(b, new, h, d).to(DTYPES[case["dtype"]])


def _plain_draw(w, u):
    """For rows of weights w in [0, 1]: the first index whose running sum, in
    units of 2^-36, passes u times the total (u in units of 2^-24); -1 for a
    row without weight.  Whole numbers: the order of the sums is of no matter."""
    w = (w.clamp(0.0, 1.0) * 2.0 ** 36).to(torch.int64)
    run = w.cumsum(-1)
    total = run[..., -1:]
    u = (u * 2.0 ** 24).to(torch.int64).clamp(0, (1 << 24) - 1)[..., None]
    point = u * (total >> 24) + ((u * (total & ((1 << 24) - 1))) >> 24)
    first = (run > point).to(torch.uint8).argmax(-1)
    return torch.where(total[..., 0] > 0, first, torch.full_like(first, -1))


def _plain_verify(s):
    case = s["case"]
    b, n = case["batch"], case["drafts"]
    tokens = s["tokens"].long()
    if case["tree"]:
        y = _plain_draw(s["p"], s["u"])                            # [b, n + 1]
        parents = s["parents"].long()
        met = tokens == y.gather(1, parents + 1)
        twin = (tokens[:, :, None] == tokens[:, None, :]) & (parents[:, :, None] == parents[:, None, :])
        met &= ~(twin & torch.ones(n, n, dtype=torch.bool, device=met.device).tril(-1)).any(-1)
        bits = torch.tensor(_tree_bits(_parents(case)), device=met.device)
        before = ((bits[:, None] >> torch.arange(n, device=met.device)) & 1) == 1
        reached = ~(before[None] & ~met[:, None, :]).any(-1)       # every draft on the path met
        count = reached.sum(-1)
        order = torch.where(reached, torch.arange(n, device=met.device), n).sort(-1).values
        last = torch.where(count > 0, order.gather(1, (count - 1).clamp_min(0)[:, None])[:, 0],
                           torch.full_like(count, -1))
        path = torch.where(order < n, order, torch.full_like(order, -1))
        return count.int(), y.gather(1, last[:, None] + 1)[:, 0].int(), path.int()
    row = torch.arange(b, device=tokens.device)
    px = s["p"][:, :n].gather(-1, tokens[..., None])[..., 0]
    qx = s["q"].gather(-1, tokens[..., None])[..., 0]
    kept = (s["u"][:, :n] * qx < px).long().cumprod(-1)
    count = kept.sum(-1)
    p = s["p"][row, count]
    q = torch.where((count < n)[:, None], s["q"][row, count.clamp_max(n - 1)], torch.zeros_like(p))
    w = (p - q).clamp_min(0.0)
    spent = ((w * 2.0 ** 36).to(torch.int64).sum(-1, keepdim=True) == 0)
    nxt = _plain_draw(torch.where(spent, p, w), s["u"][:, n])
    return count.int(), nxt.int()


# -------------------------------------------------------------------- run --

def _own(s):
    rq, case, op = _rq(), s["case"], s["case"]["op"]
    if op == "qkv":
        rq.rq_qkv_to_cache(s["layer"], s["q_in"], s["k_in"], s["v_in"], s["positions"], s["q_out"],
                           s["cache"], s["slots"], case["tokens"])
        if case["format"] == "i8":
            rq.rq_kv_read(s["cache"], s["slots"], s["k_back"], s["v_back"], case["tokens"])
    elif op == "kv_write":
        rq.rq_kv_write(s["cache"], s["k_in"], s["v_in"], s["slots"], case["tokens"])
    elif op == "kv_read":
        rq.rq_kv_read(s["cache"], s["slots"], s["k_out"], s["v_out"], case["tokens"])
    elif op == "attention":
        s["ctx"].rq_cache_attention(s["cache"], s["q"], s["out"], s["table"], s["lengths"],
                                    case["batch"], case["new"], case["q_heads"], s["scale"],
                                    tree=s["tree"])
    elif case["tree"]:
        rq.rq_verify_tree(s["tokens"], s["parents"], s["p"], s["u"], s["accepted"], s["next"],
                          s["path"], case["batch"], case["drafts"], case["vocab"])
    else:
        rq.rq_verify_chain(s["tokens"], s["p"], s["q"], s["u"], s["accepted"], s["next"],
                           case["batch"], case["drafts"], case["vocab"])


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        _own(s)
    if op == "attention":
        return s["out"] if own else _plain_attention(s)
    if op == "verify":
        if not own:
            return _plain_verify(s)
        return (s["accepted"], s["next"], s["path"]) if case["tree"] else (s["accepted"], s["next"])
    if op == "kv_read":
        return (s["k_out"], s["v_out"]) if own else _plain_rows(s)
    q = s.get("q_out") if own else _plain_rows(s)
    if op == "kv_write":
        return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if case["format"] == "i8":
        # what the integers stand for, read back in 16 bits
        k, v = (s["k_back"], s["v_back"]) if own else (x.bfloat16() for x in _plain_load(s, s["slots"]))
    else:
        k, v = s["k"], s["v"]
    return {"q": q, "k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]}


# ---------------------------------------------- the definition in 64 bits --

def _exact_rows(case, s):
    if case["op"] == "kv_read":
        out = []
        for c, sc in (("k", "ks"), ("v", "vs")):
            rows = (s[c].float().double() * s[sc].double()[..., None]).transpose(1, 2)
            out.append(rows.reshape(-1, case["kv_heads"], case["head_dim"])[s["slots"]])
        return tuple(out)
    top = TOP[case["format"]]

    def scales(x, into):
        flat = torch.zeros_like(into, dtype=torch.float64).transpose(1, 2).reshape(-1, case["kv_heads"])
        flat[s["slots"]] = x.abs().amax(-1) / top
        pages = into.shape[0]
        return flat.view(pages, case["page"], case["kv_heads"]).transpose(1, 2).contiguous()

    k, v = s["k_in"].double(), s["v_in"].double()
    if case["op"] == "kv_write":
        return {"k": None, "v": None, "k_scale": scales(k, s["ks"]), "v_scale": scales(v, s["vs"])}

    def turn(x, weight):
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
        r = case["rotary"]
        # pairs of coordinates as complex numbers, turned by the angle
        z = y[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else \
            y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
        at = s["positions"].long()
        by = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, y[..., r:]], -1)

    q, k = turn(s["q_in"].double(), s["qw"]), turn(k, s["kw"])
    # codes fall to one side or the other of a tie by the last bit of k: no 64-bit value
    return {"q": q, "k": None, "v": None, "k_scale": scales(k, s["ks"]), "v_scale": scales(v, s["vs"])}


def _exact_attention(case, s):
    d, group, new = case["head_dim"], case["q_heads"] // case["kv_heads"], case["new"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(_lengths(case)):
        pages = s["table"][i, :-(-(n + new) // case["page"])].long()

        def rows(c, sc):
            x = s[c].view(torch.uint8)[pages].view(s[c].dtype).float().double() * s[sc][pages].double()[..., None]
            return x.transpose(0, 1).flatten(1, 2)[:, :n + new]    # [kv_heads, n + new, d]

        k, v = rows("k", "ks"), rows("v", "vs")
        open_ = torch.zeros((new, n + new), dtype=torch.bool)
        open_[:, :n] = True
        if case["tree"]:
            for j, p in enumerate(_parents(case)):
                if p >= 0:
                    open_[j, n:] = open_[p, n:]
                open_[j, n + j] = True
        else:
            open_[:, n:] = torch.ones(new, new).tril().bool()
        bar = torch.where(open_, 0.0, -math.inf).double().to(k.device)
        for head in range(case["q_heads"]):
            a = s["q"][i, :, head].double() @ k[head // group].T * s["scale"] + bar
            out[i, :, head] = torch.softmax(a, -1) @ v[head // group]
    return out


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "verify":
        return None                                                # whole numbers
    return _exact_rows(case, s)
