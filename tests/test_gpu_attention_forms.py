"""GPU: what rq_cache_attention promises, on the kernel for few query rows per
kv head and on the tcgen05 kernel for many alike.  Which one runs is a matter
of sizes, the room of the page table among them; every test here asserts it."""
import pytest
import torch

from serving_util import attention, gen, random_pool, values
from test_gpu_attention import Case, random_tree, signed

pytestmark = pytest.mark.gpu
FORMS = pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
TYPES = [("f32", 0), ("f32", 1), ("f16", 0), ("f16", 1), ("bf16", 0), ("bf16", 1)]


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


@pytest.fixture(scope="module")
def ctx(rq):
    c = rq.Context()
    yield c
    c.close()


def run(ctx, c, many, q=None):
    """The case's output from the kernel for many rows (a table with room for
    the work that it starts at) or from the other (the table as it is)."""
    if many:
        hk = c.k.shape[1]
        rows = c.new * (c.hq // hk)
        room = -(-3400000 // (hk * len(c.lengths) * rows * c.page)) + 1
        if c.table.shape[1] < room:
            table = torch.full((len(c.lengths), room), -9, dtype=torch.int32)
            table[:, :c.table.shape[1]] = c.table
            c.table = table
    few0, many0 = ctx.attention_launches()
    got = c.run(ctx, q=q)
    few1, many1 = ctx.attention_launches()
    assert (few1 - few0, many1 - many0) == ((0, 1) if many else (1, 0))
    return got


@FORMS
@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads", [(6, 2, 64), (10, 2, 128)], ids=str)
@pytest.mark.parametrize("mask,new,page", [("chain", 13, 16), ("tree", 29, 32),
                                           ("prompt", 77, 256), ("prompt", 70, 128)])
def test_types_and_masks(rq, ctx, mask, new, page, heads, dtype, fmt, many):
    lengths = [130, 0, -1, 61]
    tree = random_tree(gen(new), len(lengths), new) if mask == "tree" else None
    c = Case(rq, 200 + new, lengths, new, *heads, dtype, fmt, page, tree=tree)
    c.spoil()
    c.check(run(ctx, c, many))
    assert rq.rq_get_device_status() == 0


@pytest.mark.parametrize("dtype,fmt", [("f32", 1), ("bf16", 0), ("f16", 1)])
@pytest.mark.parametrize("new,heads", [
    (32, (1, 1, 64)), (33, (2, 2, 128)), (64, (1, 1, 128)), (16, (7, 1, 64)), (18, (7, 1, 128)),
    (127, (1, 1, 128)), (128, (1, 1, 64)), (129, (1, 1, 128)), (51, (5, 1, 64)),
    (64, (4, 1, 128)), (257, (1, 1, 64)), (39, (10, 1, 128)), (55, (7, 1, 64))])
def test_partial_tiles(rq, ctx, new, heads, dtype, fmt):
    """32 .. 390 rows in tiles of 128, two to a segment."""
    c = Case(rq, 300 + new, [100, 7], new, *heads, dtype, fmt, 64)
    c.spoil()
    c.check(run(ctx, c, True))
    assert rq.rq_get_device_status() == 0


@pytest.mark.parametrize("dtype,fmt", [("f32", 1), ("f16", 0), ("bf16", 1)])
@pytest.mark.parametrize("lengths,new,heads,tree", [
    ([1500] * 30, 8, (16, 4, 64), False),          # whole segments, a thread block each
    ([1500] * 35, 16, (4, 2, 128), True),          # equal parts
    ([2900, 40, 1100, 0, 17], 24, (6, 2, 128), True),   # runs of cost
    ([290 - 5 * i for i in range(50)], 9, (16, 4, 64), False),   # several whole segments
    ([900], 600, (2, 1, 128), False), ([60, 700], 333, (4, 2, 64), False)])   # prompts
def test_cuts(rq, ctx, lengths, new, heads, tree, dtype, fmt):
    words = random_tree(gen(3), len(lengths), new) if tree else None
    c = Case(rq, 400 + new, lengths, new, *heads, dtype, fmt, 32, tree=words)
    c.spoil()
    got = run(ctx, c, True)
    c.check(got)
    assert torch.equal(run(ctx, c, True), got)
    assert rq.rq_get_device_status() == 0


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing_are_zero(rq, ctx, d, dtype, many):
    new = 20
    tree = torch.zeros((2, new), dtype=torch.int64)
    tree[1, 4] = signed(1 << 2)
    c = Case(rq, 5, [0, 0], new, 14, 2, d, dtype, 0, 16, tree=tree)
    got = run(ctx, c, many)
    c.check(got)
    got[1, 4] = 0
    assert not got.any()


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bits_past_the_new_tokens_are_ignored(rq, ctx, dtype, many):
    new = 11
    words = [(2 << i) - 1 for i in range(new)]
    c = Case(rq, 9, [50], new, 12, 2, 64, dtype, 1, 16, tree=torch.tensor([words]))
    want = run(ctx, c, many)
    c.tree = torch.tensor([[signed(w | (1 << 64) - (1 << new + i % 3)) for i, w in enumerate(words)]])
    assert torch.equal(run(ctx, c, many), want)


@FORMS
@pytest.mark.parametrize("dtype,fmt", [("f32", 0), ("f16", 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_chain_of_drafts_is_a_tree_of_one_branch(rq, ctx, d, dtype, fmt, many):
    new = 17
    c = Case(rq, 3, [333, 20], new, 14, 2, d, dtype, fmt, 64)
    chain = run(ctx, c, many)
    c.tree = torch.tensor([[(2 << i) - 1 for i in range(new)]] * 2, dtype=torch.int64)
    assert torch.equal(run(ctx, c, many), chain)
    c.check(chain)


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_not_finite_queries_stay_in_their_rows(rq, ctx, d, dtype, many):
    c = Case(rq, 8, [100], 9, 8, 2, d, dtype, 0, 16)
    want = run(ctx, c, many)
    c.q[0, 1, 3, 5] = float("inf")
    c.q[0, 2, 0, 0] = float("nan")
    c.q[0, 8, 7, d - 1] = float("-inf")
    got = run(ctx, c, many)
    bad = torch.isnan(got).all(-1)[0]
    assert bad[1, 3] and bad[2, 0] and bad[8, 7] and int(bad.sum()) == 3
    same = ~bad[None, ..., None].expand_as(got)
    assert torch.equal(got[same], want[same])


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_q(rq, ctx, dtype, many):
    c = Case(rq, 21, [200, 30], 12, 6, 2, 128, dtype, 0, 16)
    want = run(ctx, c, many)
    wide = torch.randn((2, 12, 10, 128)).to(c.q.dtype).cuda()
    wide[:, :, 2:8] = c.q.cuda()
    assert torch.equal(run(ctx, c, many, q=wide[:, :, 2:8]), want)


@FORMS
@pytest.mark.parametrize("q_scale", [1e-12, 30.0, 1e6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ranges_of_q(rq, ctx, dtype, q_scale, many):
    c = Case(rq, 77, [300, 90], 9, 8, 2, 64, dtype, 1, 32, q_scale=q_scale)
    c.vs *= torch.exp(torch.randn(c.vs.shape, generator=gen(1)))
    c.check(run(ctx, c, many))


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing_are_zero_whatever_their_queries(rq, ctx, d, bad, dtype, many):
    """Unused sequences, and rows under empty mask words, of queries that nobody
    wrote; rows between them that see something are NaN or not by their own."""
    new = 20
    tree = torch.zeros((3, new), dtype=torch.int64)
    tree[2, 5] = tree[2, 6] = 1
    c = Case(rq, 5, [0, -1, 0], new, 14, 2, d, dtype, 0, 16, tree=tree)
    finite = c.q[2, 5].clone()
    c.q[:] = float(bad)
    c.q[2, 5] = finite
    got = run(ctx, c, many)
    assert bool(torch.isnan(got[2, 6]).all()) and bool(torch.isfinite(got[2, 5]).all())
    got[2, 5:7] = 0
    assert not got.any()
    c.tree = None                      # every row sees the tokens before it
    c.lengths[0] = -3
    got = run(ctx, c, many)
    assert not got[:2].any()
    assert bool(torch.isnan(got[2, :5]).all()) and bool(torch.isnan(got[2, 6:]).all())
    assert bool(torch.isfinite(got[2, 5]).all())


def test_largest_finite_queries(rq, ctx):
    """Up to the largest f32: one key takes all, and nothing is NaN.  (The kernel
    for few rows takes differences of scores before it scales them; the other
    one's scores have to stay in f32's range, as the header says.)"""
    c = Case(rq, 6, [60], 9, 8, 2, 64, "f32", 1, 16)
    c.q[0, 4, 2] *= 3.4028e38 / float(c.q[0, 4, 2].abs().max())
    c.q[0, 5, 1] = torch.finfo(torch.float32).max
    assert bool(torch.isfinite(c.q).all()) and float(c.q[0, 4, 2].abs().max()) > 3.4e38
    assert bool(torch.isfinite(run(ctx, c, False)).all())


def test_one_head_of_256_keeps_the_same_rules(rq, ctx):
    tree = torch.zeros((2, 3), dtype=torch.int64)
    c = Case(rq, 7, [0, -1], 3, 2, 1, 256, "bf16", 0, 16, tree=tree)
    for bad in ("nan", "inf"):
        c.q[:] = float(bad)
        assert not run(ctx, c, False).any()
    c.tree = None
    assert bool(torch.isnan(run(ctx, c, False)[0]).all())


def spoil_codes(c, sequence, place):
    """NaN codes of both signs at one place of the cache."""
    page, offset = int(c.table[sequence, place // c.page]), place % c.page
    for codes in (c.k, c.v):
        row = codes.view(torch.uint8)[page, :, offset]
        row[:, 0::3] = 0x7F
        row[:, 1::3] = 0xFF


HIDDEN = [("f32", 64), ("f32", 128), ("f16", 64), ("bf16", 128)]


@FORMS
@pytest.mark.parametrize("dtype,d", HIDDEN)
def test_codes_under_cleared_bits_do_not_reach_the_output(rq, ctx, d, dtype, many):
    """NaN codes where drafts were never written: under bits that no row sets,
    and under bits that some rows set, whose own output they may spoil."""
    new = 22
    words = [((1 << new) - 1) & ~(1 << 3) & ~(1 << 17) for _ in range(new)]
    c = Case(rq, 11, [100, 0, 63], new, 14, 2, d, dtype, 0, 16, tree=torch.tensor([words] * 3))
    want = run(ctx, c, many)
    c.check(want)
    for b, n in enumerate(c.lengths.tolist()):
        spoil_codes(c, b, n + 3)
        spoil_codes(c, b, n + 17)
    assert torch.equal(run(ctx, c, many), want)
    c.tree[:, 9] |= 1 << 17
    got = run(ctx, c, many)
    got[:, 9] = want[:, 9]
    assert torch.equal(got, want)


@FORMS
@pytest.mark.parametrize("dtype,d", HIDDEN)
@pytest.mark.parametrize("new", [21, 75])
def test_codes_of_later_tokens_do_not_reach_earlier_ones(rq, ctx, new, d, dtype, many):
    c = Case(rq, 12, [100, 0], new, 10, 2, d, dtype, 0, 32)
    want = run(ctx, c, many)
    for b, n in enumerate(c.lengths.tolist()):
        for place in (n + new - 1, n + new - 4):
            spoil_codes(c, b, place)
    got = run(ctx, c, many)
    assert torch.equal(got[:, :new - 4], want[:, :new - 4])


def test_hidden_codes_at_head_size_256(rq, ctx):
    c = Case(rq, 13, [50, 0], 5, 4, 1, 256, "f32", 0, 16)
    want = run(ctx, c, False)
    for b, n in enumerate(c.lengths.tolist()):
        spoil_codes(c, b, n + 3)
    assert torch.equal(run(ctx, c, False)[:, :3], want[:, :3])


SCALES = [1e30, 1e6, 30.0, float("nan"), float("inf"), -1e30, -float("inf"), 3e38]


def spoil_scales(c, sequence, place, k_scale, v_scale):
    page, offset = int(c.table[sequence, place // c.page]), place % c.page
    c.ks[page, :, offset], c.vs[page, :, offset] = k_scale, v_scale


@FORMS
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype,fmt,d", [("f32", 0, 64), ("f32", 1, 128), ("bf16", 0, 128)])
def test_scales_under_cleared_bits_do_not_reach_the_output(rq, ctx, d, dtype, fmt, scale, many):
    """Large and odd scales under bits that no row sets, and under bits that
    one row sets: the bits of all other rows stay."""
    new = 26
    words = [((1 << new) - 1) & ~(1 << 2) & ~(1 << 17) for _ in range(new)]
    c = Case(rq, 14, [100, 0, 63], new, 14, 2, d, dtype, fmt, 16, tree=torch.tensor([words] * 3))
    want = run(ctx, c, many)
    c.check(want)
    for b, n in enumerate(c.lengths.tolist()):
        spoil_scales(c, b, n + 2, scale, scale)
        spoil_scales(c, b, n + 17, scale, scale)
    assert torch.equal(run(ctx, c, many), want)
    c.tree[:, 9] |= 1 << 2
    got = run(ctx, c, many)
    got[:, 9] = want[:, 9]
    assert torch.equal(got, want)


@FORMS
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("new,dtype,d", [(21, "f32", 128), (75, "bf16", 64), (140, "f32", 64)])
def test_scales_of_later_tokens_do_not_reach_earlier_ones(rq, ctx, new, dtype, d, scale, many):
    c = Case(rq, 15, [100, 0], new, 4, 2, d, dtype, 1, 32)
    want = run(ctx, c, many)
    c.check(want)
    for b, n in enumerate(c.lengths.tolist()):
        for i in (new - 9, new - 2):
            spoil_scales(c, b, n + i, scale, scale)
    got = run(ctx, c, many)
    assert torch.equal(got[:, :new - 9], want[:, :new - 9])


@FORMS
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rows_see_values_of_very_different_scales(rq, ctx, dtype, many):
    """Some rows see a value of scale 1e9, those beside them do not: each is
    within its own bound."""
    new = 24
    tree = torch.tensor([[(1 << new) - 1 if i % 3 == 0 else ((1 << new) - 1) & ~(1 << 5)
                          for i in range(new)]])
    c = Case(rq, 16, [90], new, 14, 2, 128, dtype, 1, 16, tree=tree)
    page, offset = int(c.table[0, 95 // 16]), 95 % 16
    c.vs[page, :, offset] = 1e9 if dtype == "f32" else 1e3
    c.check(run(ctx, c, many))


def test_hidden_scales_at_head_size_256(rq, ctx):
    for scale in SCALES:
        c = Case(rq, 17, [50, 0], 5, 4, 1, 256, "f32", 0, 16)
        want = run(ctx, c, False)
        for b, n in enumerate(c.lengths.tolist()):
            spoil_scales(c, b, n + 3, scale, scale)
        assert torch.equal(run(ctx, c, False)[:, :3], want[:, :3])


@pytest.mark.parametrize("heads,page,batch", [
    ((4, 1, 64), 256, 1025), ((4, 1, 128), 128, 1025), ((4, 1, 256), 256, 1025),
    ((8, 1, 128), 64, 40), ((2, 1, 256), 16, 40), ((28, 4, 128), 64, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_long_sums_of_few_rows(rq, ctx, heads, page, batch, fmt):
    # The tensor cores cut sums off: at most 2^-23 of the sum at each of the 2
    # additions of a unit of 16 keys, on average half of that, in the 16 units
    # that are summed there before a rounded addition (32 x 2^-24), and D / 8
    # such additions in a score of magnitude up to about 4 whose partial sums
    # are half of it on average (D / 4 x 2^-24).  More than 1024 sequences are
    # not cut; all of them read the same pages.
    hq, hk, d = heads
    n = 60000
    pages = -(-(n + 1) // page)
    k, v, ks, vs = random_pool(18, pages, hk, page, d, fmt)
    cache = rq.KVCache.from_tensors(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), format=fmt)
    table = torch.randperm(pages, generator=gen(19)).int()[None].expand(batch, -1).contiguous()
    lengths = torch.full((batch,), n, dtype=torch.int32)
    q = torch.randn((batch, 1, hq, d), generator=gen(20))
    out = torch.empty_like(q, device="cuda")
    few0, _ = ctx.attention_launches()
    ctx.rq_cache_attention(cache, q.cuda(), out, table.cuda(), lengths.cuda(), batch, 1, hq,
                           d ** -0.5)
    assert ctx.attention_launches()[0] == few0 + 1
    pick = torch.tensor(sorted({0, batch // 2, batch - 1}))
    ref, _ = attention(q[pick], values(k, ks), values(v, vs), table[pick], lengths[pick], None,
                       d ** -0.5, "f32", page)
    err = float((out.cpu().double()[pick] - ref).norm() / ref.norm())
    print("relative error %.2e, bound %.2e" % (err, (32 + d / 4) * 2.0 ** -24))
    assert err <= (32 + d / 4) * 2.0 ** -24
