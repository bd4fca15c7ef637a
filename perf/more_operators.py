"""The steps of a decoding pass between the quantized linears, as measurable cases.

Four operators: the cache slots, positions and page tables of a pass's new
tokens from the requests' lengths ("plan"), the norm after a block, the gated
and scaled residual sum and the norm before the next block ("norm"), the FP8
product with bias, activation, multiplication and residual in its epilogue
("product"), and the way from logits to tokens or to the filtered
probabilities that the verification of drafts takes ("sample", "probs").

With `own` false, run() computes a case with elementary torch operations; with
`own` true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
UNIT = 2.0 ** 42            # a token's weight is a whole number of this part of the likeliest one's


def _rq():
    import quantized_linear_layers_gb300 as rq
    return rq


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the next token of one conversation: latency counts
        dict(name="plan_one", op="plan", batch=1, new=1, context=3000, page=64, table=2048,
             packed=False),
        # a serving batch of single tokens, every sixteenth of them on a new page
        dict(name="plan_decode", op="plan", batch=256, new=1, context=30000, page=16, table=2048,
             packed=False),
        # prompts of unequal length packed one behind another, in a buffer with room
        dict(name="plan_prompts", op="plan", batch=48, new=4096, context=600, page=16, table=512,
             packed=True),
        # one token between two blocks of a layer, norms on both sides
        dict(name="norm_one", op="norm", tokens=1, width=3584, dtype="f32", residual="f32",
             post=True, gate="none", absmax=False),
        # drafted tokens of a 16-bit model with a 32-bit residual stream, odd
        # width, each channel with its own gate
        dict(name="norm_drafts", op="norm", tokens=200, width=4099, dtype="bf16", residual="f32",
             post=True, gate="channel", absmax=False),
        # the longest prefill, with the next product's absolute maximum
        dict(name="norm_prompt", op="norm", tokens=4096, width=3584, dtype="f32", residual="f32",
             post=True, gate="none", absmax=True),
        # the gate product of one token, times the up product
        dict(name="product_one", op="product", tokens=1, rows=18944, inner=3584, dtype="bf16",
             act="silu", bias=False, mul=True, residual=False, packed=False),
        # the down product of drafts onto a 32-bit residual stream
        dict(name="product_drafts", op="product", tokens=48, rows=3584, inner=18944, dtype="f32",
             act="none", bias=True, mul=False, residual=True, packed=False),
        # the gate product of a prompt
        dict(name="product_prompt", op="product", tokens=2048, rows=18944, inner=3584, dtype="bf16",
             act="silu", bias=False, mul=True, residual=False, packed=True),
        # one conversation's next token with every filter on
        dict(name="sample_one", op="sample", rows=1, vocab=131072, dtype="f32", filters="all"),
        # a serving batch whose requests ask for different filters
        dict(name="sample_batch", op="sample", rows=64, vocab=131072, dtype="f32", filters="mixed"),
        # the target's probabilities of drafted chains, nucleus only, odd vocabulary
        dict(name="probs_chains", op="probs", rows=256, vocab=50001, dtype="bf16", filters="p"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "norm", "norm", "product", "product", "sample", "sample", "probs"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    if op == "plan":
        page = rng.choice([16, 32, 64, 128, 256])
        packed = rng.random() < 0.5
        batch = _log(rng, 1, 400)
        new = _log(rng, 1, max(1, min(4096, 150000 // batch)))
        context = _log(rng, 1, 20000)
        return dict(op=op, batch=batch, new=new, context=context, page=page,
                    table=-(-(context + new) // page) + rng.randint(0, 40), packed=packed)
    if op == "norm":
        width = _log(rng, 32, 16384)
        width = width // 8 * 8 if rng.random() < 0.6 else width
        tokens = _log(rng, 1, max(1, min(4096, 4096 * 3584 // width)))
        return dict(op=op, tokens=tokens, width=width, dtype=dtype,
                    residual=rng.choice([dtype, "f32"]), post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token"]),
                    absmax=dtype == "f32" and rng.random() < 0.5)
    if op == "product":
        inner = 128 * _log(rng, 2, 148)
        rows = _log(rng, 64, 18944)
        rows = rows // 8 * 8 if rng.random() < 0.7 else rows
        tokens = _log(rng, 1, 2048)
        act = rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"])
        while tokens * rows * inner > 2048 * 18944 * 3584:
            tokens = tokens // 2
        return dict(op=op, tokens=tokens, rows=rows, inner=inner, dtype=dtype, act=act,
                    bias=rng.random() < 0.5, mul=rng.random() < 0.5, residual=rng.random() < 0.5,
                    packed=rng.random() < 0.4)
    vocab = _log(rng, 1000, 200000)
    rows = _log(rng, 1, max(1, min(256, 8000000 // vocab)))
    return dict(op=op, rows=rows, vocab=vocab, dtype=dtype,
                filters=rng.choice(["none", "k", "p", "min", "all", "mixed", "greedy"]))


def _counts(case):
    """New tokens of each sequence: the case's, or packed prompts of unequal length."""
    b, n = case["batch"], case["new"]
    return [n - (n // 2) * ((5 * i) % b) // b for i in range(b)] if case["packed"] else [n] * b


def _contexts(case):
    """Cached tokens of each sequence, from half the longest on; every eleventh place unused."""
    b, c = case["batch"], case["context"]
    return [-1 if i % 11 == 10 else c - (c // 2) * ((7 * i) % b) // b for i in range(b)]


def _plan_rows(case):
    """Rows of the pass: the padded batch, or room for the packed prompts and some more."""
    return sum(_counts(case)) + (37 if case["packed"] else 0)


def work(case):
    op = case["op"]
    if op == "plan":
        page, read, taken, live = case["page"], 0, 0, 0
        for n, c in zip(_contexts(case), _counts(case)):
            if n >= 0:
                have, all_ = -(-n // page), -(-(n + c) // page)
                taken += all_ - have
                read += all_ - n // page
                live += c
        rows = _plan_rows(case)
        return {"bytes": case["batch"] * 12 + rows * 16 + 4 * read + 4 * taken, "flops": 4 * rows}
    if op == "norm":
        n, w, r = case["tokens"] * case["width"], WIDTH[case["dtype"]], WIDTH[case["residual"]]
        gate = {"none": 0, "channel": case["width"] * w, "token": n * w}[case["gate"]]
        return {"bytes": n * (2 * w + 2 * r) + gate + (8 if case["post"] else 4) * case["width"],
                "flops": (11 if case["post"] else 7) * n}
    if op == "product":
        m, n, k, w = case["tokens"], case["rows"], case["inner"], WIDTH[case["dtype"]]
        outs = 1 + int(case["mul"]) + int(case["residual"])
        return {"bytes": m * k + n * k + outs * m * n * w + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (WIDTH[case["dtype"]] + (4 if op == "probs" else 0)), "flops": 6 * n}


# ----------------------------------------------------------------- inputs --

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _prepare_plan(case, seed, device):
    g = _gen(seed, device)
    b, page = case["batch"], case["page"]
    contexts, counts = _contexts(case), _counts(case)
    have = [max(0, -(-n // page)) for n in contexts]
    need = [max(0, -(-(n + c) // page)) - h for n, c, h in zip(contexts, counts, have)]
    pages = sum(have) + sum(need) + 50
    order = torch.randperm(pages, generator=g, device=device).to(torch.int32)
    s = dict(case=case)
    # the pages of the cached tokens, found by the table only
    held = torch.tensor(have, device=device)[:, None]
    col = torch.arange(case["table"], device=device)
    first = held.cumsum(0) - held
    s["table"] = torch.where(col < held, order[(first + col).clamp_max(pages - 1)],
                             torch.zeros((), dtype=torch.int32, device=device)).contiguous()
    s["free"] = order[sum(have):].contiguous()
    s["free_count"] = torch.tensor([pages - sum(have)], dtype=torch.int32, device=device)
    s["lengths"] = torch.tensor(contexts, dtype=torch.int32, device=device)
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device=device)
    rows = _plan_rows(case)
    s["slot"] = torch.empty(rows, dtype=torch.int64, device=device)
    s["position"] = torch.empty(rows, dtype=torch.int32, device=device)
    s["sequence"] = torch.empty(rows, dtype=torch.int32, device=device)
    s["next"] = torch.empty(b, dtype=torch.int32, device=device)
    s["left"] = torch.empty(1, dtype=torch.int32, device=device)
    return s


def _prepare_norm(case, seed, device):
    g = _gen(seed, device)
    t, w = case["tokens"], case["width"]

    def rows(dtype, spread):
        # N(0, 1) with a few strong channels, as hidden states have
        x = torch.randn((t, w), generator=g, device=device)
        x = x * (1.0 + 15.0 * (torch.rand(w, generator=g, device=device) < 0.003))
        return (spread * x).to(DTYPES[dtype])

    s = dict(case=case, y=rows(case["dtype"], 1.7), h=rows(case["residual"], 3.0))
    s["post_weight"] = 1.0 + 0.2 * torch.randn(w, generator=g, device=device)
    s["pre_weight"] = 1.0 + 0.2 * torch.randn(w, generator=g, device=device)
    s["gate"] = None
    if case["gate"] != "none":
        n = t if case["gate"] == "token" else 1
        s["gate"] = torch.randn((n, w), generator=g, device=device).to(DTYPES[case["dtype"]])
        s["gate"] = s["gate"] if n > 1 or case["gate"] == "token" else s["gate"][0]
    s["scale"] = 0.7
    s["h_out"] = torch.empty_like(s["h"])
    s["x"] = torch.empty_like(s["y"])
    s["absmax"] = torch.zeros(1, dtype=torch.int32, device=device)
    if own:
        s["layer"] = _rq().NormParams(w, post=case["post"], pre=True,
                                      post_weight=s["post_weight"] if case["post"] else None,
                                      pre_weight=s["pre_weight"], eps=EPS, scale=s["scale"])
    return s


def _codes(x):
    """E4M3 codes of x and the factor that turns them back."""
    a = x.abs().amax()
    return (x * (448.0 / a)).to(torch.float8_e4m3fn), (a / 448.0).reshape(1)


def _prepare_product(case, seed, device):
    g = _gen(seed, device)
    m, n, k = case["tokens"], case["rows"], case["inner"]
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    x = torch.zeros((-(-m // 16) * 16, k), device=device)
    x[:m] = torch.randn((m, k), generator=g, device=device)
    x[:m] *= 1.0 + 9.0 * (torch.rand(k, generator=g, device=device) < 0.002)
    s["x"], s["x_scale"] = _codes(x)
    s["w"], s["w_scale"] = _codes(torch.randn((n, k), generator=g, device=device) * k ** -0.5)
    s["bias"] = 0.3 * torch.randn(n, generator=g, device=device) if case["bias"] else None

    def rows():
        # a tensor of its own, or the second half of each row of a wider one
        if not case["packed"]:
            return torch.randn((m, n), generator=g, device=device).to(dt)
        return torch.randn((m, 2 * n), generator=g, device=device).to(dt)[:, n:]

    s["mul"] = rows() if case["mul"] else None
    s["residual"] = rows() if case["residual"] else None
    s["y"] = torch.empty((m, n), dtype=dt, device=device)
    return s


def _prepare_sample(case, seed, device):
    g = _gen(seed, device)
    r, v = case["rows"], case["vocab"]
    s = dict(case=case)
    s["logits"] = (2.5 * torch.randn((r, v), generator=g, device=device)).to(DTYPES[case["dtype"]])

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(r, generator=g, device=device)

    temperature, top_p, min_p = uniform(0.5, 1.2), uniform(0.7, 0.98), uniform(0.01, 0.1)
    top_k = torch.randint(1, 400, (r,), generator=g, device=device, dtype=torch.int32)
    which = torch.randint(0, 6, (r,), generator=g, device=device)
    s["u"] = torch.rand(r, generator=g, device=device)
    f = case["filters"]
    if f == "mixed":
        # each request asks for something else: 0 nothing, 1 top-k, 2 top-p,
        # 3 min-p, 4 all, 5 the likeliest token
        top_k = torch.where((which == 1) | (which == 4), top_k, torch.zeros_like(top_k))
        top_p = torch.where((which == 2) | (which == 4), top_p, torch.ones_like(top_p))
        min_p = torch.where((which == 3) | (which == 4), min_p, torch.zeros_like(min_p))
        temperature = torch.where(which == 5, torch.zeros_like(temperature), temperature)
    s["temperature"] = torch.zeros_like(temperature) if f == "greedy" else temperature
    s["top_k"] = top_k if f in ("k", "all", "mixed") else None
    s["top_p"] = top_p if f in ("p", "all", "mixed") else None
    s["min_p"] = min_p if f in ("min", "all", "mixed") else None
    if case["op"] == "probs":
        s["p"] = torch.empty((r, v), device=device)
    else:
        s["token"] = torch.empty(r, dtype=torch.int32, device=device)
    return s


PREPARE = {"plan": _prepare_plan, "norm": _prepare_norm, "product": _prepare_product,
           "sample": _prepare_sample, "probs": _prepare_sample}


def prepare(case, seed):
    return PREPARE[case["op"]](case, seed, torch.device("cuda"))


# ------------------------------------------------- the operators in torch --

def _plain_plan(s):
    case = s["case"]
    page = case["page"]
    length = s["lengths"].long()
    live = length >= 0
    count = torch.where(live, s["counts"].long(), torch.zeros_like(length))
    have = (length.clamp_min(0) + page - 1) // page
    need = torch.where(live, (length + count + page - 1) // page - have, torch.zeros_like(have))
    first = need.cumsum(0) - need
    left = s["free_count"].long() - need.sum()
    col = torch.arange(case["table"], device=length.device)
    new = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (s["free_count"].long() - 1 - (first[:, None] + col - have[:, None])).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(new, s["free"][at], s["table"]))
    row = torch.arange(_plan_rows(case), device=length.device)
    if case["packed"]:
        end = count.cumsum(0)
        seq = torch.searchsorted(end, row, right=True).clamp_max(case["batch"] - 1)
        i = row - (end - count)[seq]
    else:
        seq, i = row // case["new"], row % case["new"]
    filled = i < count[seq]
    place = torch.where(filled, length[seq] + i, torch.zeros_like(i))
    slot = s["table"].long()[seq, place // page] * page + place % page
    none = torch.full_like(slot, -1)
    return {"table": s["table"], "slot": torch.where(filled, slot, none), "position": place.int(),
            "sequence": torch.where(filled, seq, none).int(), "next": (length + count).int(),
            "left": left.int()}


def _plain_rms(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _plain_norm(s):
    case = s["case"]
    y = s["y"].float()
    if case["post"]:
        y = _plain_rms(y, s["post_weight"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["h"].float() + s["scale"] * y
    x = _plain_rms(h, s["pre_weight"])
    out = {"h": h.to(s["h"].dtype), "x": x.to(s["y"].dtype)}
    if case["absmax"]:
        out["absmax"] = x.abs().amax().reshape(1)
    return out


def _plain_act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z.clamp_min(0.0) if act == "relu" else z


def _plain_product(s):
    case = s["case"]
    z = torch.matmul(s["x"][:case["tokens"]].float(), s["w"].float().T) * (s["x_scale"] * s["w_scale"])
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _plain_act(z, case["act"])
    if s["mul"] is not None:
        z = z * s["mul"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(DTYPES[case["dtype"]])


def _plain_kept(s):
    """Whole-number weights of the tokens, zero where a filter takes them out:
    64 bits, since a running sum falls to one side or the other of a border."""
    logits = s["logits"].float()
    best = logits.amax(-1, keepdim=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    far = (logits.double() - best.double()) / torch.where(greedy, torch.ones_like(t), t)
    weight = torch.floor(torch.exp(far) * UNIT).long()
    value, order = logits.sort(dim=-1, descending=True, stable=True)
    weight = weight.gather(-1, order)
    stays = weight > 0
    stays &= ~greedy | (torch.arange(weight.shape[-1], device=weight.device) == 0)
    if s["min_p"] is not None:
        stays &= weight >= torch.ceil(s["min_p"].double() * UNIT).long()[:, None]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        stays &= (stays.long().cumsum(-1) <= k) | (k <= 0)
    if s["top_p"] is not None:
        weight = torch.where(stays, weight, torch.zeros_like(weight))
        run = weight.cumsum(-1)
        p = s["top_p"].double()[:, None]
        most = torch.ceil(p * run[:, -1:].double()).long().clamp_min(1)
        stays &= (run - weight < most) | (p >= 1)
    weight = torch.where(stays, weight, torch.zeros_like(weight))
    return torch.zeros_like(weight).scatter_(-1, order, weight)


def _plain_sample(s):
    weight = _plain_kept(s)
    run = weight.cumsum(-1)
    total = run[:, -1:]
    if s["case"]["op"] == "probs":
        return (weight.double() / total.double()).float()
    u = (s["u"] * 2.0 ** 24).long().clamp(0, (1 << 24) - 1)[:, None]
    point = u * (total >> 24) + ((u * (total & ((1 << 24) - 1))) >> 24)
    return (run > point).to(torch.uint8).argmax(-1).int()


# -------------------------------------------------------------------- run --

def _own(s):
    rq, case, op = _rq(), s["case"], s["case"]["op"]
    if op == "plan":
        rq.rq_batch_plan(s["lengths"], s["table"], s["free"], s["free_count"], s["left"], s["slot"],
                         s["position"], case["page"], count=s["counts"],
                         new_tokens=0 if case["packed"] else case["new"], sequence=s["sequence"],
                         next_length=s["next"])
        return {"table": s["table"], "slot": s["slot"], "position": s["position"],
                "sequence": s["sequence"], "next": s["next"], "left": s["left"]}
    if op == "norm":
        rq.rq_residual_norm(s["layer"], s["y"], s["h"], s["h_out"], s["x"], case["tokens"],
                            gate=s["gate"], absmax_bits=s["absmax"] if case["absmax"] else None)
        out = {"h": s["h_out"], "x": s["x"]}
        if case["absmax"]:
            out["absmax"] = s["absmax"].view(torch.float32)
        return out
    if op == "product":
        rq.rq_fp8_gemm_epilogue(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], case["tokens"],
                                case["rows"], case["inner"], act=case["act"], bias=s["bias"],
                                mul=s["mul"], residual=s["residual"])
        return s["y"]
    filters = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if op == "probs":
        rq.rq_token_probs(s["logits"], s["p"], case["rows"], case["vocab"], **filters)
        return s["p"]
    rq.rq_sample(s["logits"], s["u"], s["token"], case["rows"], case["vocab"], **filters)
    return s["token"]


PLAIN = {"plan": _plain_plan, "norm": _plain_norm, "product": _plain_product,
         "sample": _plain_sample, "probs": _plain_sample}


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ---------------------------------------------- the definition in 64 bits --

def _exact_norm(case, s):
    def unit(x):
        return x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["width"] + EPS)

    y = s["y"].double()
    if case["post"]:
        y = unit(y) * s["post_weight"].double()
    if case["gate"] != "none":
        y = y * s["gate"].double()
    # the scale is a 32-bit number
    h = torch.add(s["h"].double(), y, alpha=float(torch.tensor(s["scale"], dtype=torch.float32)))
    x = unit(h) * s["pre_weight"].double()
    out = {"h": h, "x": x}
    if case["absmax"]:
        out["absmax"] = torch.linalg.vector_norm(x, math.inf).reshape(1)
    return out


def _exact_product(case, s):
    z = torch.einsum("mk,nk->mn", s["x"][:case["tokens"]].float().double(), s["w"].float().double())
    z = z * s["x_scale"].double() * s["w_scale"].double()
    if case["bias"]:
        z = z + s["bias"].double()
    if case["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif case["act"] == "gelu":
        z = z * torch.special.ndtr(z)
    elif case["act"] == "gelu_tanh":
        # (1 + tanh a) / 2 is the logistic function of 2 a
        z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif case["act"] == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    if case["mul"]:
        z = z * s["mul"].double()
    return z + s["residual"].double() if case["residual"] else z


def _exact_probs(case, s):
    logits, t = s["logits"].double(), s["temperature"].double()[:, None]
    order = torch.argsort(-logits, dim=-1, stable=True)            # likeliest first, equal ones by index
    p = torch.softmax(logits / torch.where(t > 0, t, torch.ones_like(t)), -1).gather(-1, order)
    # how many of that order stay
    n = torch.where(t > 0, case["vocab"], 1)
    if s["min_p"] is not None:
        n = torch.minimum(n, (p >= s["min_p"].double()[:, None] * p[:, :1]).sum(-1, keepdim=True))
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        n = torch.where(k > 0, torch.minimum(n, k), n)
    rank = torch.arange(case["vocab"], device=n.device)
    p = torch.where(rank < n, p, torch.zeros_like(p))
    if s["top_p"] is not None:
        top = s["top_p"].double()[:, None]
        upto = p.cumsum(-1) / p.sum(-1, keepdim=True)
        m = 1 + torch.searchsorted(upto, top.contiguous())         # the first whose sum reaches it, and those before
        p = torch.where((rank < m) | (top >= 1), p, torch.zeros_like(p))
    return torch.zeros_like(p).scatter_(-1, order, p / p.sum(-1, keepdim=True))


def exact(case, seed):
    global own
    if case["op"] in ("plan", "sample"):
        return None                                                # whole numbers
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm": _exact_norm, "product": _exact_product, "probs": _exact_probs}[case["op"]](case, s)
