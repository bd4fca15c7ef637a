"""GPU: attention over the paged quantized cache against its definition in 64
bits, within the bound that serving_util.attention derives per output."""
import pytest
import torch

from serving_util import TORCH, attention, encode, gen, random_pool, values

pytestmark = pytest.mark.gpu
SENTINEL = 0x7FC0DEAD


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def signed(w):
    return w - (1 << 64) if w >> 63 else w


def random_tree(g, b, new, empty=False):
    """Ancestor masks of random trees; with `empty`, some rows see no draft."""
    rows = []
    for _ in range(b):
        words = []
        for i in range(new):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            words.append((1 << i) | (words[p] if p >= 0 else 0))
        if empty:
            words = [0 if i % 3 == 0 else w for i, w in enumerate(words)]
        rows.append([signed(w) for w in words])
    return torch.tensor(rows, dtype=torch.int64)


class Case:
    def __init__(self, rq, seed, lengths, new, hq, hk, d, dtype, fmt, page, tree=None, spare=3,
                 q_scale=1.0):
        g = gen(seed)
        b = len(lengths)
        self.rq, self.new, self.hq, self.dtype, self.page = rq, new, hq, dtype, page
        need = [max(0, -(-(n + new) // page)) if n >= 0 else 0 for n in lengths]
        pages = sum(need) + spare
        self.k, self.v, self.ks, self.vs = random_pool(seed, pages, hk, page, d, fmt)
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((b, max(need + [1]) + 1), -9, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n].int()
            at += n
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.q = (q_scale * torch.randn((b, new, hq, d), generator=g)).to(TORCH[dtype])
        self.tree = tree
        self.scale = d ** -0.5
        self.fmt = fmt

    def spoil(self):
        """What no row may see: places behind a sequence's last one and the
        unused pages get NaN codes and NaN scales."""
        live = torch.zeros(self.ks.shape, dtype=torch.bool)
        for i, n in enumerate(self.lengths.tolist()):
            for p in range(max(0, n + self.new) if n >= 0 else 0):
                live[self.table[i, p // self.page], :, p % self.page] = True
        self.k.view(torch.uint8)[~live] = 0x7F
        self.v.view(torch.uint8)[~live] = 0xFF
        self.ks[~live] = float("nan")
        self.vs[~live] = float("nan")

    def run(self, ctx, q=None):
        rq = self.rq
        cache = rq.KVCache.from_tensors(self.k.cuda(), self.v.cuda(), self.ks.cuda(),
                                        self.vs.cuda(), format=self.fmt)
        q = self.q.cuda() if q is None else q
        words = self.q.numel() * self.q.element_size() // 4
        buf = torch.full((words + 2048,), SENTINEL, dtype=torch.int32, device="cuda")
        out = buf[1024:1024 + words].view(TORCH[self.dtype]).view(self.q.shape)
        tree = None if self.tree is None else self.tree.cuda()
        ctx.rq_cache_attention(cache, q, out, self.table.cuda(), self.lengths.cuda(),
                               len(self.lengths), self.new, self.hq, self.scale, tree=tree)
        assert bool((buf[:1024] == SENTINEL).all()) and bool((buf[-1024:] == SENTINEL).all())
        return out.cpu()

    def check(self, got):
        ref, tol = attention(self.q, values(self.k, self.ks), values(self.v, self.vs), self.table,
                             self.lengths, self.tree, self.scale, self.dtype, self.page)
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-300)).max())


@pytest.fixture(scope="module")
def ctx(rq):
    c = rq.Context()
    yield c
    c.close()


HEADS = [(28, 4, 128), (8, 8, 64), (4, 1, 256), (16, 2, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lengths,page", [
    ([0], 16),                       # the first token of all
    ([15], 16), ([63], 64), ([64], 64), ([1000], 32),
    ([1, 700, -1, 0, 129], 128),     # ragged, with an unused sequence
])
def test_single_tokens(rq, ctx, lengths, page, heads, fmt, dtype):
    c = Case(rq, 7 * len(lengths) + lengths[0], lengths, 1, *heads, dtype, fmt, page)
    c.spoil()
    c.check(c.run(ctx))
    assert rq.rq_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,new,lengths,page", [
    ((28, 4, 128), 64, [100, 0], 16), ((28, 4, 128), 13, [63, 500, 64, -1], 64),
    ((5, 5, 64), 3, [126], 128), ((8, 1, 256), 33, [40], 32), ((40, 8, 64), 2, [10, 11, 12], 16)])
def test_trees(rq, ctx, heads, new, lengths, page, fmt, dtype):
    g = gen(new)
    for empty in (False, True):
        tree = random_tree(g, len(lengths), new, empty)
        c = Case(rq, 100 + new, lengths, new, *heads, dtype, fmt, page, tree=tree)
        c.spoil()
        c.check(c.run(ctx))
    assert rq.rq_get_device_status() == 0


def test_rows_that_see_nothing_are_zero(rq, ctx):
    """No cached token and an empty mask word; a NaN under every cleared bit."""
    new = 20
    tree = torch.zeros((2, new), dtype=torch.int64)
    tree[1, 4] = signed(1 << 2)
    for dtype in ("f32", "f16"):
        c = Case(rq, 5, [0, 0], new, 14, 2, 64, dtype, 0, 16, tree=tree)
        keep = (int(c.table[1, 0]), 2)
        ks, vs = c.ks[keep[0], :, keep[1]].clone(), c.vs[keep[0], :, keep[1]].clone()
        c.ks[:], c.vs[:] = float("nan"), float("inf")
        c.ks[keep[0], :, keep[1]], c.vs[keep[0], :, keep[1]] = ks, vs
        got = c.run(ctx)
        live = got[1, 4].clone()
        got[1, 4] = 0
        assert not got.any()
        want = values(c.v, c.vs)[keep[0], :, keep[1]].repeat_interleave(7, 0)
        assert bool(((live.double() - want).abs() <= 2.0 ** -10 * want.abs() + 1e-7).all())


def test_bits_past_the_new_tokens_are_ignored(rq, ctx):
    tree = torch.tensor([[1, 3, 7]], dtype=torch.int64)
    c = Case(rq, 9, [50], 3, 4, 2, 64, "f32", 1, 16, tree=tree)
    want = c.run(ctx)
    c.tree = torch.tensor([[signed(1 | ~7 & (1 << 64) - 1), 3 | 1 << 40, signed(7 | 1 << 63)]],
                          dtype=torch.int64)
    assert torch.equal(c.run(ctx), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,new,lengths", [
    ((28, 4, 128), 70, [0, 3]), ((6, 2, 64), 200, [129]), ((2, 1, 256), 131, [60]),
    ((4, 4, 128), 65, [0, 700, -1])])
def test_prompts(rq, ctx, heads, new, lengths, dtype):
    c = Case(rq, 40 + new, lengths, new, *heads, dtype, new % 2, 64)
    c.spoil()
    c.check(c.run(ctx))
    assert rq.rq_get_device_status() == 0


def test_chain_of_drafts_is_a_tree_of_one_branch(rq, ctx):
    new = 17
    c = Case(rq, 3, [333, 20], new, 28, 4, 128, "f32", 0, 64)
    chain = c.run(ctx)
    c.tree = torch.tensor([[(2 << i) - 1 for i in range(new)]] * 2, dtype=torch.int64)
    assert torch.equal(c.run(ctx), chain)
    c.check(chain)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequence_is_split_and_joined(rq, ctx, dtype):
    """One long sequence over all SMs beside short ones; equal calls, equal bits."""
    c = Case(rq, 12, [20011, 5, 3000], 2, 14, 2, 128, dtype, 0, 64)
    got = c.run(ctx)
    c.check(got)
    for _ in range(3):
        assert torch.equal(c.run(ctx), got)
    fresh = rq.Context()
    assert torch.equal(c.run(fresh), got)
    fresh.close()


@pytest.mark.parametrize("q_scale", [1e-12, 30.0, 1e6])
def test_ranges_of_q(rq, ctx, q_scale):
    """Tiny queries (a plain mean), sharp ones, and ones so sharp that a row
    is one key; scales of rows far apart."""
    for dtype in ("f32", "bf16"):
        c = Case(rq, 77, [300, 90], 3, 8, 2, 64, dtype, 1, 32, q_scale=q_scale)
        c.vs *= torch.exp(3 * torch.randn(c.vs.shape, generator=gen(1)))
        c.check(c.run(ctx))


def test_not_finite_queries_stay_in_their_rows(rq, ctx):
    c = Case(rq, 8, [100], 4, 8, 2, 64, "f32", 0, 16)
    want = c.run(ctx)
    c.q[0, 1, 3, 5] = float("inf")
    c.q[0, 2, 0, 0] = float("nan")
    got = c.run(ctx)
    bad = torch.isnan(got).all(-1)[0]
    assert bad[1, 3] and bad[2, 0] and int(bad.sum()) == 2
    same = ~bad[None, ..., None].expand_as(got)
    assert torch.equal(got[same], want[same])


def test_strided_q(rq, ctx):
    c = Case(rq, 21, [200, 30], 5, 6, 2, 128, "bf16", 0, 16)
    want = c.run(ctx)
    wide = torch.randn((2, 5, 10, 128)).bfloat16().cuda()
    wide[:, :, 2:8] = c.q.cuda()
    assert torch.equal(c.run(ctx, q=wide[:, :, 2:8]), want)


def test_indexes_outside_are_reported(rq, ctx):
    c = Case(rq, 33, [100, 40], 1, 4, 2, 64, "f32", 0, 16)
    assert rq.rq_get_device_status() == 0
    want = c.run(ctx)
    table = c.table.clone()
    c.table[0, 2] = 1 << 30
    got = c.run(ctx)
    assert rq.rq_get_device_status() == 9
    assert torch.equal(got[1], want[1])
    c.table[0, 2] = -1
    c.run(ctx)
    assert rq.rq_get_device_status() == 9
    c.table = table
    c.lengths = torch.tensor([1 << 30, 40], dtype=torch.int32)   # past the page table
    got = c.run(ctx)
    assert rq.rq_get_device_status() == 9
    assert torch.equal(got[1], want[1])
    assert torch.equal(c.run(ctx)[1], want[1])
    assert rq.rq_get_device_status() == 9


def test_cache_past_32_bit_offsets(rq, ctx):
    """The same sequence at the front and past 2^32 bytes of a cache."""
    hk, d, page, fmt = 8, 256, 256, 1
    pages = (1 << 32) // (hk * d * page) + 3
    cache = rq.KVCache(pages, page, hk, d, fmt)
    k, v, ks, vs = (x.cuda() for x in random_pool(4, 2, hk, page, d, fmt))
    outs = []
    q = torch.randn((1, 1, hk, d), device="cuda")
    for at in (0, pages - 2):
        for dst, src in ((cache.k, k), (cache.v, v), (cache.k_scale, ks), (cache.v_scale, vs)):
            dst.zero_()
            dst[at:at + 2].copy_(src)
        table = torch.tensor([[at, at + 1]], dtype=torch.int32, device="cuda")
        n = torch.tensor([400], dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        ctx.rq_cache_attention(cache, q, out, table, n, 1, 1, hk, 0.05)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and bool(outs[0].any())
    assert rq.rq_get_device_status() == 0
    del cache
    torch.cuda.empty_cache()


def test_other_stream_and_graph(rq):
    own = rq.Context()
    c = Case(rq, 50, [2000, 100], 1, 14, 2, 64, "f32", 0, 64)
    cache = rq.KVCache.from_tensors(c.k.cuda(), c.v.cuda(), c.ks.cuda(), c.vs.cuda())
    q, table, n = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    out = torch.empty_like(q)

    def call():
        own.rq_cache_attention(cache, q, out, table, n, 2, 1, 14, c.scale)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()                                   # the scratch is allocated here
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for i in range(2):
        c.q = torch.randn(c.q.shape, generator=gen(i))
        q.copy_(c.q)
        n.copy_(torch.tensor([1500 + i, 99 + i], dtype=torch.int32))
        c.lengths = n.cpu()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out.cpu())
    own.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,long", [(77, 1150), (90, 1300), (130, 2000), (200, 3000)])
def test_one_longer_sequence_among_many_short_ones(rq, ctx, batch, long, dtype):
    """Runs of cost that are shorter than a unit somewhere; every part counted
    in a join has to be there."""
    lengths = [i % 9 for i in range(batch)]
    lengths[batch // 3] = long
    c = Case(rq, batch, lengths, 1, 4, 1, 128, dtype, 0, 16)
    c.spoil()
    got = c.run(ctx)
    c.check(got)
    assert torch.equal(c.run(ctx), got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,new,heads", [
    ([5000, 3, 900, 40, 2500], 40, (28, 4, 128)),      # two row tiles, one of them half empty
    ([12000], 64, (8, 1, 128)), ([3000, 2900, 700], 19, (14, 2, 64))])
def test_shared_segments_of_many_rows(rq, ctx, lengths, new, heads, dtype):
    g = gen(new)
    c = Case(rq, new, lengths, new, *heads, dtype, 0, 64, tree=random_tree(g, len(lengths), new))
    c.spoil()
    got = c.run(ctx)
    c.check(got)
    for _ in range(2):
        assert torch.equal(c.run(ctx), got)
    assert rq.rq_get_device_status() == 0


def test_long_sums_of_many_rows(rq, ctx):
    # The tensor cores cut sums off: at most 2^-23 of the sum at each of the 8
    # additions of a unit of 64 keys, on average half of that, in the 6 units
    # that are summed there before a rounded addition (2.9e-6); 16 in a score
    # of magnitude up to about 4, half of them small (1.9e-6).
    g = gen(77)
    c = Case(rq, 77, [8000] * 8, 48, 28, 4, 128, "f32", 0, 64, tree=random_tree(g, 8, 48))
    got = c.run(ctx).double()[:1]
    ref, _ = attention(c.q[:1], values(c.k, c.ks), values(c.v, c.vs), c.table[:1], c.lengths[:1],
                       c.tree[:1], c.scale, c.dtype, c.page)
    assert float((got - ref).norm() / ref.norm()) <= 4.8e-6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,new,heads", [(1100, 1, (2, 1, 64)), (300, 160, (8, 1, 64))])
def test_more_tiles_than_are_cut_by_length(rq, ctx, batch, new, heads, dtype):
    lengths = [(37 * i) % 90 for i in range(batch)]
    lengths[7], lengths[batch - 1], lengths[20] = 900, 700, -1
    c = Case(rq, 78, lengths, new, *heads, dtype, 0, 64)
    got = c.run(ctx).double()
    sel = torch.tensor([0, 1, 7, 20, 21, batch // 2, batch - 1])
    ref, tol = attention(c.q[sel], values(c.k, c.ks), values(c.v, c.vs), c.table[sel],
                         c.lengths[sel], None, c.scale, c.dtype, c.page)
    assert bool(((got[sel] - ref).abs() <= tol).all())
    assert bool((c.run(ctx).double() == got).all())
    assert rq.rq_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,new,lengths", [
    ((4, 1, 256), 1, [8000]), ((8, 1, 256), 1, [40000]), ((8, 1, 256), 6, [40000]),
    ((4, 1, 128), 1, [40000]), ((3, 1, 64), 1, [60000])])
def test_joins_of_more_than_one_level(rq, ctx, heads, new, lengths, fmt, dtype):
    """One sequence in more than 8 parts: groups of neighbours are joined, then
    the groups.  At head size 256 two warps share a row of the join."""
    c = Case(rq, 90 + new, lengths, new, *heads, dtype, fmt, 64)
    c.spoil()
    got = c.run(ctx)
    c.check(got)
    for _ in range(4):
        assert torch.equal(c.run(ctx), got)
    assert rq.rq_get_device_status() == 0


def test_scratch_stays_where_a_captured_graph_uses_it(rq):
    """Single tokens are captured; then the context serves a prompt of many
    rows, and what the allocator has to give is overwritten."""
    own = rq.Context()
    c = Case(rq, 51, [6000, 100], 1, 14, 2, 64, "f32", 0, 64)
    cache = rq.KVCache.from_tensors(c.k.cuda(), c.v.cuda(), c.ks.cuda(), c.vs.cuda())
    q, table, n = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    out = torch.empty_like(q)

    def call():
        own.rq_cache_attention(cache, q, out, table, n, 2, 1, 14, c.scale)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    prompt = Case(rq, 52, [3000, 700], 40, 28, 4, 128, "f32", 0, 64)
    prompt.check(prompt.run(own))
    batch = Case(rq, 53, [500 + 7 * i for i in range(90)], 1, 32, 8, 128, "bf16", 0, 64)
    batch.run(own)
    spoiled = [torch.full((1 << 24,), float("nan"), device="cuda") for _ in range(4)]
    for i in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out.cpu())
    assert all(bool(torch.isnan(x).all()) for x in spoiled)
    own.close()


def test_first_call_inside_a_capture_is_refused(rq):
    own = rq.Context()
    c = Case(rq, 54, [70], 1, 4, 2, 64, "f32", 0, 16)
    cache = rq.KVCache.from_tensors(c.k.cuda(), c.v.cuda(), c.ks.cuda(), c.vs.cuda())
    q, table, n = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(rq.RqError) as e:
            own.rq_cache_attention(cache, q, out, table, n, 1, 1, 4, c.scale)
        assert e.value.status == 5
        out += 1.0                               # the capture goes on
    graph.replay()
    torch.cuda.synchronize()
    assert bool((out == 1.0).all())
    c.check(c.run(own))
    own.close()
