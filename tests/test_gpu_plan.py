"""GPU: a pass's slots, positions and page tables against one token after
another in Python."""
import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(rq, length, count, new_tokens, page, max_pages, spare=5, rows=None, free_count=None,
          table=None, seed=0):
    """Runs the plan on random tables and compares everything that it writes."""
    g = ref.gen(seed)
    batch = len(length)
    live = [n if n >= 0 else 0 for n in length]
    c = [new_tokens] * batch if count is None else [max(0, x) for x in count]
    need = sum(-(-(n + x) // page) for n, x in zip(live, c)) + spare
    order = torch.randperm(need + batch * max_pages, generator=g).tolist()
    free = order[:need]
    if table is None:
        rest = order[need:]
        table = [[rest[b * max_pages + j] for j in range(max_pages)] for b in range(batch)]
    free_count = len(free) if free_count is None else free_count
    if rows is None:
        rows = batch * new_tokens if new_tokens else sum(x for n, x in zip(length, c) if n >= 0)
    want = ref.plan(length, count, new_tokens, page, table, free, free_count, rows)
    t = i32(table).reshape(batch, max_pages)
    slot = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    position, sequence = i32([88] * rows), i32([99] * rows)
    left, start, following = i32([-5]), i32([0] * (batch + 1)), i32([0] * batch)
    rq.rq_batch_plan(i32(length), t, i32(free), i32([free_count]), left, slot, position, page,
                     count=None if count is None else i32(count), new_tokens=new_tokens,
                     sequence=sequence, row_start=start, next_length=following)
    status = rq.rq_get_device_status()
    assert slot.tolist() == want["slot"]
    assert position.tolist() == want["position"]
    assert sequence.tolist() == want["sequence"]
    assert t.tolist() == want["table"]
    assert left.tolist() == [want["left"]]
    assert start.tolist() == want["start"]
    assert following.tolist() == want["next"]
    assert status == (9 if want["bad"] else 0)
    return want


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 255, 256, 700])
def test_one_sequence(rq, page, length):
    for new in (1, 2, 17, 300):
        check(rq, [length], None, new, page, 64)
        check(rq, [length], [new], 0, page, 64)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("batch", [2, 33, 257, 1025, 3000])
def test_batches_of_unequal_sequences(rq, batch, packed):
    g = ref.gen(batch)
    length = torch.randint(-20, 200, (batch,), generator=g).clamp_min(-1).tolist()
    count = torch.randint(-1, 8, (batch,), generator=g).clamp_min(-1).tolist()
    count = [0 if i % 5 == 0 else x for i, x in enumerate(count)]
    check(rq, length, count, 0 if packed else 7, 16, 14)


def test_long_prompts_over_several_blocks(rq):
    check(rq, [5, -1, 0, 1000, 31], [3000, 50, 1, 2047, 4096], 0, 32, 200)
    check(rq, [5, -1, 0, 1000, 31], [1500, 50, 1, 0, 3], 1500, 32, 200)


def test_rows_without_tokens(rq):
    want = check(rq, [3, -1, 60], [2, 4, 0], 4, 16, 8)
    assert want["slot"][2:] == [-1] * 10
    # a packed buffer with room, no tokens at all, and no sequences
    check(rq, [3, -1, 60], [2, 4, 5], 0, 16, 8, rows=1500)
    check(rq, [3, 4], [0, 0], 0, 16, 8, rows=3)
    check(rq, [-1, -1], None, 3, 16, 8)


def test_what_does_not_fit_is_recorded(rq):
    # counts above the rows of a sequence; packed tokens without a row
    assert check(rq, [3, 5], [9, 2], 4, 16, 8)["bad"]
    assert check(rq, [3, 5, 9], [9, 2, 4], 0, 16, 8, rows=10)["bad"]
    # a stack that does not hold enough, or nothing; more than it can hold
    assert check(rq, [16, 16, 16], None, 20, 16, 8, free_count=3)["left"] == -3
    assert check(rq, [16, 16], None, 1, 16, 8, free_count=0)["bad"]
    assert check(rq, [16, 16], None, 1, 16, 8, free_count=-4)["bad"]
    assert check(rq, [16, 16], None, 1, 16, 8, free_count=1 << 30)["bad"]
    # past the table, from the first token and from a later one
    assert check(rq, [128, 120], None, 20, 16, 8)["bad"]
    # an entry that names no page
    assert check(rq, [3], None, 2, 16, 2, table=[[-1, 7]])["bad"]
    # and nothing is left recorded behind
    assert not check(rq, [3], None, 2, 16, 2)["bad"]


def test_places_at_the_end_of_32_bits(rq):
    n = 0x7FFFFFFF
    table, free = i32([[4, 5]]), i32([1, 2])
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    position, following = i32([0, 0]), i32([0])
    rq.rq_batch_plan(i32([n]), table, free, i32([2]), i32([0]), slot, position, 16, new_tokens=2,
                     next_length=following)
    assert rq.rq_get_device_status() == 9
    assert slot.tolist() == [-1, -1] and following.tolist() == [n]
    assert position.tolist() == [n, n] and table.tolist() == [[4, 5]]


def test_slots_past_32_bits(rq):
    slot = torch.zeros(3, dtype=torch.int64, device="cuda")
    rq.rq_batch_plan(i32([255]), i32([[2000000000, 0]]), i32([2100000000]), i32([1]), i32([0]), slot,
                     i32([0] * 3), 256, new_tokens=3)
    assert slot.tolist() == [2000000000 * 256 + 255, 2100000000 * 256, 2100000000 * 256 + 1]
    assert rq.rq_get_device_status() == 0


def test_the_largest_batch(rq):
    batch = 65536
    length = [(i * 37) % 50 for i in range(batch)]
    check(rq, length, None, 1, 16, 4, spare=0)


def test_optional_outputs_may_be_left_out(rq):
    slot, position = torch.zeros(2, dtype=torch.int64, device="cuda"), i32([0, 0])
    rq.rq_batch_plan(i32([0, 16]), i32([[9, 9], [8, 9]]), i32([3, 4]), i32([2]), i32([0]), slot,
                     position, 16, new_tokens=1)
    assert slot.tolist() == [4 * 16, 3 * 16] and position.tolist() == [0, 16]


def test_replayed_passes_continue_each_other(rq):
    # lengths and the stack's count go back and forth between two buffers
    length, following = i32([0, 14, 31]), i32([0, 0, 0])
    count, left = i32([40]), i32([0])
    free = i32(list(range(100, 140)))
    table = i32([[0] * 8, [7] + [0] * 7, [5, 6] + [0] * 6])
    slot, position = torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0] * 3)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            rq.rq_batch_plan(length, table, free, count, left, slot, position, 16, new_tokens=1,
                             next_length=following)
            rq.rq_batch_plan(following, table, free, left, count, slot, position, 16,
                             new_tokens=1, next_length=length)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert length.tolist() == [40, 54, 71]
    assert count.tolist() == [40 - 3 - 3 - 3]
    used = [table.tolist()[b][:-(-n // 16)] for b, n in enumerate([40, 54, 71])]
    assert len({p for r in used for p in r}) == sum(len(r) for r in used)
    assert position.tolist() == [39, 53, 70]
    assert slot.tolist() == [used[b][n // 16] * 16 + n % 16 for b, n in enumerate([39, 53, 70])]
    assert rq.rq_get_device_status() == 0
