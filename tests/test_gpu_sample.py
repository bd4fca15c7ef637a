"""GPU: tokens and filtered probabilities from logits, against whole-number
weights on the CPU."""
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


def run(rq, logits, u=None, t=None, k=None, p=None, m=None, dtype=None):
    """(tokens for u, probabilities) of rows of logits (a tensor on the GPU)."""
    rows, vocab = logits.shape
    args = dict(temperature=None if t is None else f32(t),
                top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda"),
                top_p=None if p is None else f32(p), min_p=None if m is None else f32(m))
    u = f32([0.5] * rows if u is None else u)
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((rows, vocab), -7.0, device="cuda")
    rq.rq_sample(logits, u, token, rows, vocab, **args)
    rq.rq_token_probs(logits, probs, rows, vocab, **args)
    assert rq.rq_get_device_status() == 0
    return token.tolist(), probs.cpu().numpy()


def check(rq, logits, u, t=None, k=None, p=None, m=None):
    """Compares both entry points with the definition.  The device's weights are
    within 2^-32 of their value and a unit of the definition's: what stands
    closer than their sum's error to a border may fall to either side, and a
    random number's point may meet either neighbour there."""
    rows, vocab = logits.shape
    tokens, probs = run(rq, logits, u, t, k, p, m)
    host = logits.float().cpu().numpy()
    for r in range(rows):
        w, near = ref.staying(host[r], 1.0 if t is None else t[r], 0 if k is None else k[r],
                              1.0 if p is None else p[r], 0.0 if m is None else m[r])
        if w is None:
            assert tokens[r] == -1 and not probs[r].any()
            continue
        got = probs[r]
        assert np.array_equal(got[~near] > 0, w[~near] > 0) or \
            (w[(got > 0) != (w > 0)] <= 2).all()
        if not near.any():
            total, slack = float(w.sum()), ref.slack_of(w)
            # the weight's own error and the total's; the power of two is
            # within 2^-22 (ex2.approx), and the correction of its argument,
            # the total's inverse and the two products round four times more:
            # 2^-22 + 4 2^-24 = 8 u
            tol = (w / 2.0 ** 32 + 2.0 + slack * (w / total)) / total + 8 * ref.U * (w / total)
            assert (np.abs(got - w / total) <= tol).all()
            want, point, run_ = ref.drawn(w, u[r])
            if tokens[r] != want:
                lo = run_[tokens[r] - 1] if tokens[r] > 0 else 0
                assert w[tokens[r]] > 0 and lo - slack <= point <= run_[tokens[r]] + slack
        else:
            assert got[tokens[r]] > 0


def uniform(g, n):
    return torch.rand(n, generator=g).tolist()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 5, 127, 1000, 4097, 32000, 50001, 131072])
def test_filters(rq, vocab, dtype):
    g = ref.gen(vocab)
    rows = 7 if vocab > 40000 else 14
    logits = (2.5 * torch.randn(rows, vocab, generator=g)).to(ref.DTYPES[dtype]).cuda()
    u = uniform(g, rows)
    t = [0.3 + 0.2 * (i % 6) for i in range(rows)]
    k = [(0, 1, 2, 50, 700, vocab, vocab + 9)[i % 7] for i in range(rows)]
    p = [(0.9, 0.5, 0.99, 0.0, 1.0, 0.01, 0.95)[i % 7] for i in range(rows)]
    m = [(0.0, 0.05, 1e-6, 1.0, 0.3, 2.0, -1.0)[i % 7] for i in range(rows)]
    check(rq, logits, u)
    check(rq, logits, u, t=t)
    check(rq, logits, u, t=t, k=k)
    check(rq, logits, u, t=t, p=p)
    check(rq, logits, u, t=t, m=m)
    check(rq, logits, u, k=k, p=p)
    check(rq, logits, u, t=t, k=k, p=p, m=m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [600, 5000, 131072])
def test_top_k_around_the_sizes_that_are_listed(rq, vocab, dtype):
    g = ref.gen(vocab + 1)
    ks = [2, 31, 32, 33, 64, 100, 120, 127, 128, 129, 200, 255, 256, 257, 400, 480, 500, 511, 512,
          513, 560, 599]
    rows = len(ks)
    logits = (2.5 * torch.randn(rows, vocab, generator=g)).to(ref.DTYPES[dtype]).cuda()
    u = uniform(g, rows)
    check(rq, logits, u, k=ks)
    check(rq, logits, u, k=ks, p=[0.8] * rows)
    check(rq, logits, u, t=[1.5] * rows, k=ks, p=[0.999] * rows, m=[0.01] * rows)
    check(rq, logits, u, k=ks, p=[0.0] * rows)


def test_likeliest(rq):
    g = ref.gen(2)
    logits = torch.randn(6, 3001, generator=g)
    logits[1, 2000] = logits[1, 700] = 50.0
    logits[2, :] = -4.0
    want = [int(r.argmax()) for r in logits]
    want[1], want[2] = 700, 0
    for t in ([0.0] * 6, [-1.0] * 6, [float("nan")] * 6):
        tokens, probs = run(rq, logits.cuda(), uniform(g, 6), t=t, p=[0.5] * 6)
        assert tokens == want
        assert np.array_equal(probs, np.eye(3001, dtype=np.float32)[want])
    tokens, _ = run(rq, logits.cuda(), uniform(g, 6), k=[1] * 6)
    assert tokens == want


@pytest.mark.parametrize("vocab", [600, 5000, 131072])
def test_equal_logits(rq, vocab):
    # more equal tokens than are listed one by one: cut by index
    logits = torch.zeros(4, vocab, device="cuda")
    logits[1, 300:] = 1.5
    logits[2, ::2] = -0.0
    logits[3, vocab // 2:] = 3.0
    for k in (2, 3, 257, vocab - 300, vocab - 299, vocab):
        check(rq, logits, [0.0, 0.3, 0.7, 0.999], k=[k] * 4)
        check(rq, logits, [0.0, 0.3, 0.7, 0.999], k=[k] * 4, p=[0.77] * 4)
    for p in (0.1, 0.5, 0.9):
        check(rq, logits, [0.1, 0.3, 0.7, 0.999], p=[p] * 4)
    _, probs = run(rq, logits, k=[300] * 4)
    assert (probs[0, :300] > 0).all() and not probs[0, 300:].any()


def test_crowded_logits(rq):
    # thousands of different logits in one bin, apart in their last bits only,
    # in one spot, in two, and around zero down to the smallest floats
    n = 30000
    g = ref.gen(3)
    one = torch.tensor(7.0).view(torch.int32) - torch.randint(0, 5000, (n,), generator=g).int()
    two = torch.where(torch.rand(n, generator=g) < 0.5, one, one - 3000000)
    tiny = torch.randint(0, 1 << 30, (n,), generator=g).int().view(torch.float32) * 1e-3
    tiny = torch.where(torch.rand(n, generator=g) < 0.5, -tiny, tiny).clamp(-0.01, 0.01)
    logits = torch.stack([one.view(torch.float32), two.view(torch.float32), tiny,
                          torch.randn(n, generator=g) * 1e-4]).cuda()
    u = uniform(g, 4)
    for k in (2, 600, 5000, 15000, 29999):
        check(rq, logits, u, k=[k] * 4)
    for p in (0.01, 0.5, 0.98):
        check(rq, logits, u, p=[p] * 4)
        check(rq, logits, u, t=[30.0] * 4, k=[9000] * 4, p=[p] * 4)


def test_weights_at_the_edges_of_their_bins(rq):
    # likely tokens at the upper edges of the 43/512 octave wide bins that
    # places are guessed by, unlikely ones at the lower edges: a nucleus that
    # ends a bin and more before the guess, and one behind it
    octaves = 43.0 / 512
    upper = torch.arange(60).double() * octaves + 0.0005
    lower = (60 + torch.arange(60).double()) * octaves + octaves - 0.0005
    y = torch.cat([torch.zeros(1).double(), upper.repeat_interleave(40), lower.repeat_interleave(160)])
    flipped = torch.cat([torch.zeros(1).double(),
                         (upper + octaves - 0.001).repeat_interleave(40),
                         (lower - octaves + 0.001).repeat_interleave(160)])
    for places in (y, flipped):
        logits = (-places * np.log(2.0)).float()
        order = torch.randperm(len(logits), generator=ref.gen(4))
        logits = logits[order][None].expand(24, -1).contiguous().cuda()
        w = ref.weights(logits[0].cpu().numpy(), 1.0).astype(np.float64)
        likely = float(w[logits[0].cpu().numpy() > -60.0 * octaves * np.log(2.0)].sum() / w.sum())
        p = [likely + 0.01 * d for d in np.linspace(-2.5, 2.5, 24)]
        check(rq, logits, uniform(ref.gen(5), 24), p=p)
        check(rq, logits, uniform(ref.gen(6), 24), p=p, k=[9000] * 24, m=[1e-6] * 24)


def test_weights_of_many_set_bits_in_one_bin(rq):
    # 2^20 tokens of one weight whose low bits are set: sums of its parts
    n = 1 << 20
    best = min((float(x) for x in np.linspace(0.5, 0.6, 20000).astype(np.float32)),
               key=lambda x: int(~ref.weights(np.array([0.0, -x], np.float32), 1.0)[1] & 0x3FFF))
    logits = torch.full((2, n), -best)
    logits[0, 77] = 0.0
    logits[1, 1 << 19] = 0.0
    check(rq, logits.cuda(), [0.25, 0.75], p=[0.5, 0.999])


def test_infinities_and_nans(rq):
    inf, nan = float("inf"), float("nan")
    rows = torch.zeros(8, 700)
    rows[0, :] = -inf
    rows[1, :] = nan
    rows[2, 5:] = -inf
    rows[3, 100:] = nan
    rows[4, 650] = inf
    rows[5, 3], rows[5, 600] = inf, inf
    rows[6, 9], rows[6, 10] = 3e38, -3e38
    rows[7, 650], rows[7, 20] = -inf, nan
    u = [0.9] * 8
    logits = rows.cuda()
    for more in (dict(), dict(k=[3] * 8), dict(p=[0.9] * 8), dict(m=[0.1] * 8),
                 dict(t=[0.0] * 8), dict(t=[inf] * 8), dict(t=[1e-30] * 8),
                 dict(t=[1e-42] * 8, p=[0.5] * 8), dict(k=[690] * 8, p=[0.9] * 8)):
        check(rq, logits, u, **more)
    # parameters that are not numbers switch their filter off
    check(rq, logits, u, p=[nan] * 8)
    tokens, _ = run(rq, logits, u, m=[nan] * 8, p=[nan] * 8, k=[-3] * 8)
    assert tokens == run(rq, logits, u)[0]
    tokens, _ = run(rq, logits, [nan] * 8)
    assert tokens[3] == 0


def test_every_random_number_meets_a_token_that_stays(rq):
    g = ref.gen(5)
    logits = torch.randn(1, 1000, generator=g).expand(64, 1000).contiguous().cuda()
    u = [0.0, 2.0 ** -25, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0] + uniform(g, 58)
    check(rq, logits, u, p=[0.6] * 64)
    tokens, probs = run(rq, logits, u, k=[7] * 64)
    assert all(probs[r, t] > 0 for r, t in enumerate(tokens))
    # 0 meets the first that stays and the largest number the last
    stays = np.flatnonzero(probs[0])
    assert tokens[0] == stays[0] and tokens[2] == tokens[3] == stays[-1]


def test_draws_follow_the_probabilities(rq):
    g = ref.gen(6)
    n = 4096
    logits = torch.randn(1, 50, generator=g).expand(n, 50).contiguous().cuda()
    tokens, probs = run(rq, logits, [(i + 0.5) / n for i in range(n)], t=[0.8] * n, p=[0.9] * n)
    seen = np.bincount(tokens, minlength=50) / n
    # evenly spaced numbers: each token's share to within one on either side
    assert np.abs(seen - probs[0]).max() <= 2.0 / n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_apart_and_unaligned(rq, dtype):
    g = ref.gen(7)
    wide = torch.randn(5, 9001, generator=g).to(ref.DTYPES[dtype]).cuda()
    for lo, hi in ((0, 8000), (1, 9001), (3, 8004), (2, 6)):
        part = wide[:, lo:hi]
        k, p = [40] * 5, [0.8] * 5
        got = run(rq, part, [0.4] * 5, k=k, p=p)
        want = run(rq, part.contiguous(), [0.4] * 5, k=k, p=p)
        assert got[0] == want[0] and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("vocab", [400000, 1 << 20])
def test_vocabularies_larger_than_shared_memory(rq, vocab):
    g = ref.gen(8)
    logits = (2 * torch.randn(3, vocab, generator=g)).cuda()
    logits[2] = 1.0
    u = [0.2, 0.6, 0.99]
    check(rq, logits, u)
    check(rq, logits, u, t=[0.7] * 3, k=[900, 300000, 70000])
    check(rq, logits, u, t=[0.7] * 3, p=[0.9, 0.3, 0.5], m=[0.0, 1e-4, 0.0])


def test_many_rows(rq):
    g = ref.gen(9)
    logits = torch.randn(3000, 300, generator=g).cuda()
    u = uniform(g, 3000)
    tokens, probs = run(rq, logits, u, k=[20] * 3000, p=[0.9] * 3000)
    again, same = run(rq, logits[:1500], u[:1500], k=[20] * 1500, p=[0.9] * 1500)
    assert tokens[:1500] == again and np.array_equal(probs[:1500], same)
    check(rq, logits[1000:1040], u[1000:1040], k=[20] * 40, p=[0.9] * 40)


def test_probabilities_feed_the_verification(rq):
    # a chain without drafts draws from p by itself, with weights of 2^-36
    g = ref.gen(10)
    rows, vocab = 64, 2000
    logits = (2 * torch.randn(rows, vocab, generator=g)).cuda()
    u = f32(uniform(g, rows))
    args = dict(temperature=f32([0.7] * rows), top_p=f32([0.9] * rows))
    token, accepted, following = (torch.empty(rows, dtype=torch.int32, device="cuda")
                                  for _ in range(3))
    p = torch.empty(rows, vocab, device="cuda")
    rq.rq_sample(logits, u, token, rows, vocab, **args)
    rq.rq_token_probs(logits, p, rows, vocab, **args)
    rq.rq_verify_chain(torch.empty(rows, 1, dtype=torch.int32, device="cuda"), p, None, u, accepted,
                       following, rows, 0, vocab)
    total = p.double().cumsum(-1)
    for r in range(rows):
        a, b = int(token[r]), int(following[r])
        if a != b:  # the point lies on the border between them, to p's own rounding
            assert abs(float(total[r, min(a, b)]) - float(u[r])) < vocab * 2.0 ** -24
    assert (token == following).float().mean() > 0.95


def test_equal_calls_in_a_graph_and_on_a_stream(rq):
    g = ref.gen(11)
    rows, vocab = 40, 50001
    logits = torch.randn(rows, vocab, generator=g).cuda()
    u, top_p = f32(uniform(g, rows)), f32([0.9] * rows)
    k = torch.full((rows,), 1000, dtype=torch.int32, device="cuda")
    out = [(torch.empty(rows, dtype=torch.int32, device="cuda"),
            torch.empty(rows, vocab, device="cuda")) for _ in range(3)]

    def call(i, **more):
        rq.rq_sample(logits, u, out[i][0], rows, vocab, top_k=k, top_p=top_p, **more)
        rq.rq_token_probs(logits, out[i][1], rows, vocab, top_k=k, top_p=top_p, **more)

    call(0)
    torch.cuda.synchronize()
    call(1, stream=torch.cuda.Stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for o in out[1:]:
        assert torch.equal(o[0], out[0][0]) and torch.equal(o[1], out[0][1])
