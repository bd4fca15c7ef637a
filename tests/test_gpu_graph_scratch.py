"""GPU: FP8 activations of captured passes.  A graph quantizes its input at every
replay, into a scratch that no later call moves, overwrites or is misled by."""
import pytest
import torch

import synthetic

pytestmark = pytest.mark.gpu
N, K = 512, 1024


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def packed(rq, seed, n, k):
    w = synthetic.weight_matrix(seed, rq.RQ_Q4K, n, k)
    return torch.from_numpy(w.view("uint8").reshape(-1).copy()).cuda()


def rows(seed, m, k):
    return torch.from_numpy(synthetic.activation(seed, m, k)).cuda()


class Pass:
    """A product of M tokens by rq_linear_epilogue (or rq_linear) from x into y."""

    def __init__(self, rq, ctx, M, plain=False):
        self.rq, self.ctx, self.M, self.plain = rq, ctx, M, plain
        self.w = packed(rq, 5, N, K)
        self.x = rows(6, M, K)
        self.y = torch.zeros(M, N, device="cuda")

    def run(self, invalidate=True):
        if invalidate:
            self.ctx.rq_act_cache_invalidate()
        if self.plain:
            self.ctx.rq_linear(self.rq.RQ_Q4K, self.w, self.x, self.y, self.M, N, K)
        else:
            self.ctx.rq_linear_epilogue(self.rq.RQ_Q4K, self.w, self.x, self.y, self.M, N, K,
                                        act="silu")

    def eager(self, seed):
        """The pass's result on rows(seed), by a context of its own."""
        ctx = self.rq.Context()
        p = Pass(self.rq, ctx, self.M, self.plain)
        p.x.copy_(rows(seed, self.M, K))
        p.run()
        torch.cuda.synchronize()
        ctx.close()
        return p.y

    def capture(self, **more):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.run(**more)
        return graph


@pytest.mark.parametrize("M", [1, 3, 20])
def test_a_longer_call_between_replays(rq, M):
    ctx = rq.Context()
    p = Pass(rq, ctx, M)
    p.run()
    graph = p.capture()
    # a prompt of the next request: its activation is larger than all before
    long = Pass(rq, ctx, 2048)
    long.run()
    torch.cuda.synchronize()
    kept = long.y.clone()
    # (what a freed scratch's place would be given to)
    junk = [torch.full((1 << 20,), 0x7E, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for seed in (31, 32):
        p.x.copy_(rows(seed, M, K))
        p.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y, p.eager(seed))
    assert all(bool((t == 0x7E).all()) for t in junk) and torch.equal(long.y, kept)
    assert rq.rq_get_device_status() == 0
    ctx.close()


@pytest.mark.parametrize("M,plain", [(1, False), (20, False), (20, True)])
def test_a_capture_quantizes_what_was_cached_before_it(rq, M, plain):
    ctx = rq.Context()
    p = Pass(rq, ctx, M, plain)
    p.run()                                   # x is cached
    graph = p.capture(invalidate=False)       # the same x, nothing invalidated
    p.x.copy_(rows(33, M, K))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.y, p.eager(33))
    ctx.close()


@pytest.mark.parametrize("M,plain", [(5, False), (20, True)])
def test_a_call_does_not_find_what_was_only_captured(rq, M, plain):
    ctx = rq.Context()
    p = Pass(rq, ctx, M, plain)
    p.run()
    graph = p.capture()
    misses = ctx.stats()["act_misses"]
    p.y.zero_()
    p.run(invalidate=False)                   # captured, but never replayed
    torch.cuda.synchronize()
    assert torch.equal(p.y, p.eager(6)) and ctx.stats()["act_misses"] == misses + 1
    # and what it cached is not what a replay quantizes afterwards
    z, out = rows(34, M, K), torch.zeros(M, N, device="cuda")
    ctx.rq_act_cache_invalidate()
    ctx.rq_linear(rq.RQ_Q4K, p.w, z, out, M, N, K)
    first = out.clone()
    p.x.copy_(rows(35, M, K))
    graph.replay()
    out.zero_()
    hits = ctx.stats()["act_hits"]
    ctx.rq_linear(rq.RQ_Q4K, p.w, z, out, M, N, K)
    torch.cuda.synchronize()
    assert ctx.stats()["act_hits"] == hits + 1
    assert torch.equal(out, first) and torch.equal(p.y, p.eager(35))
    ctx.close()


def test_calls_of_one_capture_share_an_activation(rq):
    ctx = rq.Context()
    p, q = Pass(rq, ctx, 20), Pass(rq, ctx, 20, plain=True)
    q.x = p.x
    p.run()
    q.run()
    stats = ctx.stats()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
        q.run(invalidate=False)
    assert ctx.stats()["act_hits"] == stats["act_hits"] + 1
    assert ctx.stats()["act_misses"] == stats["act_misses"] + 1
    p.x.copy_(rows(36, 20, K))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.y, p.eager(36)) and torch.equal(q.y, q.eager(36))
    ctx.close()


def test_graphs_of_growing_size_and_their_replays(rq):
    # each capture needs a larger scratch than the one before, and allocates it
    ctx = rq.Context()
    passes = [Pass(rq, ctx, m) for m in (1, 17, 40, 300)]
    passes[0].run()                           # (the weight's FP8 form)
    for p in passes[1:]:
        p.w = passes[0].w
    graphs = [p.capture() for p in passes]
    for seed in (37, 38):
        for i in (3, 0, 2, 1, 0, 3):
            p = passes[i]
            p.x.copy_(rows(seed + i, p.M, K))
            p.y.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(p.y, p.eager(seed + i))
    assert rq.rq_get_device_status() == 0
    ctx.close()
