"""GPU: which tokens the filters leave, checked against a definition that knows
every token's own weight, and what is drawn and written of just those."""
import math

import numpy as np
import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def run(rq, logits, u, t=None, k=None, p=None, m=None):
    rows, vocab = logits.shape
    args = dict(temperature=None if t is None else f32(t),
                top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda"),
                top_p=None if p is None else f32(p), min_p=None if m is None else f32(m))
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((rows, vocab), -7.0, device="cuda")
    rq.rq_sample(logits, f32(u), token, rows, vocab, **args)
    rq.rq_token_probs(logits, probs, rows, vocab, **args)
    assert rq.rq_get_device_status() == 0
    return token.tolist(), probs.cpu().numpy()


def check(rq, logits, u, t=None, k=None, p=None, m=None):
    """A token may be on the other side of a cut than the definition has it only
    if it is near that cut, or if its weight is one that the device may round to
    none (1) or to one (0).  What the device keeps is then the ground on which
    its probabilities and its draw are compared.  Rows whose weights are exact
    (all logits that weigh anything equal to the largest) have nothing near.
    Returns how many tokens were on the other side."""
    rows, vocab = logits.shape
    tokens, probs = run(rq, logits, u, t, k, p, m)
    host = logits.float().cpu().numpy()
    crossed = 0
    for r in range(rows):
        temp = 1.0 if t is None else t[r]
        w, near = ref.staying(host[r], temp, 0 if k is None else k[r], 1.0 if p is None else p[r],
                              0.0 if m is None else m[r])
        if w is None:
            assert tokens[r] == -1 and not probs[r].any()
            continue
        whole = ref.weights(host[r], max(temp, 2.0 ** -116) if temp > 0 else 1.0)
        exact = bool(((whole == 0) | (whole == ref.UNIT)).all()) and not \
            (np.abs(host[r][whole == 0]) < np.inf).any()
        got = probs[r]
        kept = got > 0
        other = kept != (w > 0)
        crossed += int(other.sum())
        may = np.zeros_like(near) if exact else near | (whole <= 1)
        assert not (other & ~may).any(), np.flatnonzero(other & ~may)[:5]
        # what is kept are the first tokens in their order
        order = np.lexsort((np.arange(vocab), -np.where(np.isnan(host[r]), -np.inf, host[r])))
        sure = kept[order][whole[order] > 1]
        assert not (sure[1:] & ~sure[:-1]).any()
        held = np.where(kept, np.maximum(whole, 1), 0)
        total, slack = int(held.sum()), 0.0 if exact else ref.slack_of(held)
        # within 2^-21 of itself (8 u), for the definition's weight, which the
        # device has to 2^-32 of it and a unit, and the same of the total
        tol = (0.0 if exact else (held / 2.0 ** 32 + 1.0 + slack * (held / total)) / total) + \
            8 * ref.U * (held / total)
        assert (np.abs(got - held / total) <= tol).all()
        want, point, run_ = ref.drawn(held, u[r])
        if tokens[r] != want:
            lo = run_[tokens[r] - 1] if tokens[r] > 0 else 0
            assert kept[tokens[r]] and lo - slack <= point <= run_[tokens[r]] + slack
            assert not exact
    return crossed


def uniform(g, n):
    return torch.rand(n, generator=g).tolist()


@pytest.mark.parametrize("vocab", [600, 5000, 131072])
def test_equal_logits_are_cut_where_the_definition_cuts_them(rq, vocab):
    # every weight is the same whole number: nothing is near a border
    logits = torch.zeros(4, vocab, device="cuda")
    logits[1, 1:] = -float("inf")
    logits[1, ::3] = 2.0
    logits[1, 1::3] = 2.0
    logits[2, ::2] = -0.0
    logits[3, : vocab // 2] = -float("inf")
    u = [0.0, 0.3, 0.7, 0.999]
    for p in (0.0, 1e-9, 0.1, 0.5, 0.75, 0.9, 0.99999):
        assert check(rq, logits, u, p=[p] * 4) == 0
        assert check(rq, logits, u, p=[p] * 4, k=[vocab // 3] * 4) == 0
        assert check(rq, logits, u, p=[p] * 4, m=[1.0] * 4) == 0
    for k in (2, 100, 128, 129, 512, 513, vocab // 2, vocab):
        assert check(rq, logits, u, k=[k] * 4) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [700, 4097, 50001, 131072])
def test_what_each_filter_leaves(rq, vocab, dtype):
    g = ref.gen(vocab + 7)
    rows = 7
    logits = (2.5 * torch.randn(rows, vocab, generator=g)).to(ref.DTYPES[dtype]).cuda()
    u = uniform(g, rows)
    t = [0.3 + 0.25 * i for i in range(rows)]
    k = [2, 40, 128, 129, 600, vocab // 2, vocab]
    p = [0.9, 0.5, 0.99, 0.0, 0.7, 0.01, 0.95]
    m = [0.0, 0.05, 1e-6, 1.0, 0.3, 1e-3, 0.02]
    for more in (dict(), dict(t=t), dict(t=t, k=k), dict(t=t, p=p), dict(t=t, m=m), dict(k=k, p=p),
                 dict(t=t, k=k, p=p, m=m)):
        check(rq, logits, u, **more)


def test_tokens_at_the_edges_of_the_finer_bins(rq):
    """A cut's bin, a 512th of 43 octaves, is divided into 128: floats on both
    sides of those edges, which one pass counts and another lists."""
    step = 43.0 / 512 / 128 * math.log(2.0)
    edges = -step * np.arange(1, 40 * 128, 7)
    near = np.concatenate([np.nextafter(np.float32(edges), np.float32(s)) for s in (-9, 9)]
                          + [np.float32(edges)])
    g = ref.gen(12)
    logits = torch.from_numpy(np.concatenate([[0.0], near]).astype(np.float32))
    logits = logits[torch.randperm(len(logits), generator=g)]
    n = len(logits)
    ks = [513 + 37 * i for i in range(43)]
    assert ks[-1] < n
    rows = logits[None].expand(len(ks), n).contiguous().cuda()
    tokens, probs = run(rq, rows, uniform(g, len(ks)), k=ks)
    for r, k in enumerate(ks):
        assert int((probs[r] > 0).sum()) == k and probs[r][tokens[r]] > 0
    check(rq, rows, uniform(g, len(ks)), k=ks)
    check(rq, rows, uniform(g, len(ks)), p=[(i + 0.5) / len(ks) for i in range(len(ks))])


def whole_number_weights(l, t):
    """2^42 e^(l / t) with its fraction, of f32 differences l and a temperature."""
    import decimal
    decimal.getcontext().prec = 40
    t = decimal.Decimal(float(np.float32(t)))
    return [decimal.Decimal(float(x)) / t for x in l], decimal.Decimal(2) ** 42


@pytest.mark.parametrize("t", [1.0, 0.7])
def test_probabilities_of_the_smallest_weights(rq, t):
    """p = W / total to 2^-21 of itself for W from 1 on, and 0 where W is 0: the
    distribution that rq_sample draws from, whatever filters are on.  Only
    weights whose value is not within a 2^-30th of a whole number are looked at,
    so that W is the same however it is evaluated (to 2^-32)."""
    g = ref.gen(13)
    l = torch.cat([torch.zeros(1), -t * (14 + 15.5 * torch.rand(6000, generator=g)),
                   -t * (27.5 + 2 * torch.rand(3000, generator=g))])
    far, unit = whole_number_weights(l.numpy(), t)
    value = [unit * x.exp() for x in far]
    whole = np.array([int(v) for v in value], dtype=np.int64)
    sure = np.array([min(v - int(v), int(v) + 1 - v) > v / 2 ** 30 for v in value])
    sure[0] = True  # the largest
    assert sure.sum() > 8000 and (whole[sure] == 0).any() and (whole[sure] == 1).any()
    logits = l[None].cuda()
    rows = []
    for more in (dict(), dict(p=[0.9999999]), dict(k=[len(l)]), dict(m=[1e-30])):
        _, probs = run(rq, logits, [0.5], t=[t], **more)
        rows.append(probs[0])
        if "p" in more:
            continue  # (the cut takes some out)
        got = probs[0].astype(np.float64)
        total = float(whole.sum())
        tol = 8 * ref.U * whole / total + 2.0 ** -149 + slack_of_total(whole, got)
        assert np.array_equal(got[sure] > 0, whole[sure] > 0)
        assert (np.abs(got - whole / total)[sure] <= tol[sure]).all()
    # a nucleus of 1 - 2^-23 has a total smaller by that, and the same weights
    kept = (rows[1] > 0) & sure
    assert (np.abs(rows[1] - rows[0])[kept] <= (2.0 ** -20 + 2.0 ** -22) * rows[0][kept]).all()


def slack_of_total(whole, got):
    """The total's own error: 2^-32 of it and a unit a token."""
    return got * (2.0 ** -32 + len(whole) / float(whole.sum()))
