"""Plain definitions of the steps between the linears, on the CPU in 64 bits
or whole numbers."""
import math

import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------- plan --

def plan(length, count, new_tokens, page, table, free, free_count, rows):
    """Everything rq_batch_plan writes, one token after another; `bad` where it
    records an index."""
    table = [list(r) for r in table]
    max_pages = len(table[0]) if table else 0
    out = dict(slot=[-1] * rows, position=[0] * rows, sequence=[-1] * rows, start=[], next=[],
               bad=False)
    top = min(max(free_count, 0), len(free))
    out["bad"] |= top != free_count
    taken, row = 0, 0
    for b, n in enumerate(length):
        c = (new_tokens if count is None else max(count[b], 0)) if n >= 0 else 0
        if new_tokens and c > new_tokens:
            c, out["bad"] = new_tokens, True
        first = b * new_tokens if new_tokens else row
        out["start"].append(min(first, rows))
        out["next"].append(n + c)
        pages = list(range(-(-max(n, 0) // page), min(-(-(n + c) // page), max_pages))) if c else []
        stack = {}
        for p in pages:
            stack[p] = free[top - 1 - taken] if top - 1 - taken >= 0 else -1
            taken += 1
        for i in range(c):
            place, r = n + i, first + i
            if r >= rows:
                out["bad"] = True
                continue
            p = place // page
            entry = -1
            if p < max_pages:
                entry = stack.get(p, table[b][p] if p not in stack else None)
                if p in stack and place % page == 0:
                    table[b][p] = entry
            out["slot"][r] = entry * page + place % page if entry >= 0 else -1
            out["bad"] |= entry < 0
            out["position"][r], out["sequence"][r] = place, b
        row += new_tokens if new_tokens else c
    out["start"].append(min(row, rows))
    out["table"], out["left"] = table, top - taken
    return out


# ------------------------------------------------------------------- norm --

def norm(y, h, post, pre, post_weight, pre_weight, gate, scale, eps, width):
    """(h', x, bounds of both before their last rounding) in 64 bits.

    Bounds, u = 2^-24: a thread adds at most 16 squares and 5 + 5 joins follow,
    so a mean square is within 28 u (with its two products), its root within
    14 u; rsqrtf is within 2 units (4 u); the products with the weight, the
    root and the gate round thrice, the last sum once."""
    h = h.double()
    eh = torch.zeros_like(h)
    if y is not None:
        t = y.double()
        if post:
            t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)
            t = t * post_weight.double() if post_weight is not None else t
        if gate is not None:
            t = t * gate.double()
        t = t * float(np.float32(scale))
        h = h + t
        eh = 22 * U * t.abs() + U * h.abs()
    if not pre:
        return h, h, eh, eh
    root = torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    w = pre_weight.double() if pre_weight is not None else torch.ones(width, dtype=torch.float64)
    rel = 20 * U + eh.norm(dim=-1, keepdim=True) / h.norm(dim=-1, keepdim=True).clamp_min(1e-300)
    x = h / root * w
    return h, x, eh, (eh / root) * w.abs() + x.abs() * rel


# ---------------------------------------------------------------- product --

def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z.clamp_min(0) if name == "relu" else z


def product(x, xs, w, ws, bias, name, mul, residual, dtype):
    """(y, bound) of E4M3 codes x [M, K], w [N, K] (as floats).

    Sums: each of the K / 32 additions to the f32 sum may cut off a unit
    (2^-23), and so may the joins of 32 products, of the sum of magnitudes; the
    scales and the bias round four times.  The activations' slopes are below
    1.13; their own evaluation is within 16 u of |z|, SiLU's fast form within
    2^-21 (1 + |z|) of its value."""
    K = x.shape[1]
    s = float(xs) * float(ws)
    z = (x.double() @ w.double().T) * s
    ez = (x.abs().double() @ w.abs().double().T) * s * (K / 32 + 8) * 2.0 ** -23 + 4 * U * z.abs()
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * z.abs()
    a = act(z, name)
    ea = 1.13 * ez
    if name != "none":
        ea = ea + 16 * U * z.abs()
        if name == "silu" and dtype != torch.float32:
            ea = ea + 2.0 ** -21 * (1 + z.abs()) * a.abs()
    y, ey = a, ea
    if mul is not None:
        y, ey = y * mul.double(), ey * mul.double().abs()
    if residual is not None:
        y = y + residual.double()
    return y, ey + ROUND[dtype] * (y.abs() + ey) + TINY[dtype]


# --------------------------------------------------------------- sampling --

UNIT = 1 << 42


def weights(logits, t):
    """Whole weights (numpy int64) of a row in 64 bits; None: nothing to draw."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return None
    with np.errstate(invalid="ignore", over="ignore"):
        far = np.where(l == top, 0.0, (l - top) / np.float64(np.float32(t)))
        far = np.where(np.isnan(far), -np.inf, far)
    return np.floor(np.exp(far) * UNIT).astype(np.int64)


def slack_of(w):
    """How far sums of the device's weights may be from the definition's: each
    is within 2^-32 of its value and one unit."""
    return int(w.sum()) / 2.0 ** 32 + len(w) + 1


def staying(logits, t=1.0, k=0, p=1.0, m=0.0):
    """(weights by index with zeros for what goes, tokens so near to a nucleus'
    or to min-p's border that they may fall to either side)."""
    if not t > 0:
        t, k = 1.0, 1
    t = max(t, 2.0 ** -116)
    w = weights(logits, t)
    if w is None:
        return None, None
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64)) + 0.0
    order = np.lexsort((np.arange(len(l)), -l))
    s = w[order]
    near = np.zeros(len(l), dtype=bool)
    slack = slack_of(w)
    if m > 0:
        least = math.ceil(min(np.float64(np.float32(m)), 1.0) * UNIT)
        near |= (np.abs(s - least) <= least / 2.0 ** 32 + 2) & (least != UNIT)
        s = np.where(s >= least, s, 0)
    if k > 0:
        s = np.where(np.cumsum(s > 0) <= k, s, 0)
    if p < 1:
        run = np.cumsum(s)
        goal = max(1, math.ceil(max(float(np.float32(p)), 0.0) * float(run[-1])))
        near |= (np.abs(run - s - goal) <= slack) & (np.arange(len(l)) > 0)
        s = np.where(run - s < goal, s, 0)
    out, close = np.zeros_like(w), np.zeros_like(near)
    out[order], close[order] = s, near
    return out, close


def drawn(w, u):
    """The token that u meets, and the point and running sums behind it."""
    run = np.cumsum(w)
    total = int(run[-1])
    u = float(np.float32(u))
    un = min(max(int(math.floor(u * 2.0 ** 24)), 0), (1 << 24) - 1) if u == u else 0
    point = un * total >> 24
    return int(np.argmax(run > point)), point, run
