"""Blocks and slots for requests, and row writes through them, on the GPU
against the plain forms (needs a GB300)."""
import numpy as np
import pytest

import _paged
from _paged import BLOCK, blocks_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


def dev(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


class Assign:
    """Device buffers of one kvtc_paged_assign call."""

    def __init__(self, kv, held, lens, free, head, table, slot_capacity,
                 in_place=False):
        import torch
        self.kv, self.R = kv, len(lens)
        self.held = dev(held, np.int32)
        self.lens = dev(lens, np.int32)
        self.free = dev(free, np.int32)
        self.head = dev([head], np.int64)
        self.table = dev(table, np.int32)
        guard = 5                      # entries behind each output
        self.slots = torch.full((slot_capacity + guard,), 77,
                                dtype=torch.int64, device="cuda")
        self.cu = torch.full((self.R + 1 + guard,), 77, dtype=torch.int64,
                             device="cuda")
        self.held_out = self.held if in_place else torch.full_like(self.held,
                                                                   77)
        self.head_out = self.head if in_place else torch.full_like(self.head,
                                                                   77)
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = kv.kvtc_paged_assign_workspace_bytes(self.R)
        self.ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        self.capacity = slot_capacity

    def call(self, flags=True):
        self.kv.kvtc_paged_assign(
            self.R, self.held, self.lens,
            self.free if self.free.numel() else None, self.free.numel(),
            self.head, self.table, self.table.shape[1], BLOCK,
            self.slots if self.capacity else None, self.capacity, self.cu,
            self.held_out, self.head_out, self.ws, self.ws.numel(),
            self.flags if flags else None)

    def check(self, ref):
        table, slots, cu, held_out, head_out, short = ref
        np.testing.assert_array_equal(self.table.cpu().numpy(), table)
        got = self.slots.cpu().numpy()
        np.testing.assert_array_equal(got[:self.capacity], slots)
        assert (got[self.capacity:] == 77).all()
        got = self.cu.cpu().numpy()
        np.testing.assert_array_equal(got[:self.R + 1], cu)
        assert (got[self.R + 1:] == 77).all()
        np.testing.assert_array_equal(self.held_out.cpu().numpy(), held_out)
        assert int(self.head_out.cpu()[0]) == head_out
        assert int(self.flags.cpu()[0]) == \
            (self.kv.KVTC_FLAG_SPACE if short else 0)


def run_assign(kv, held, lens, free, head, table, slot_capacity, **more):
    c = Assign(kv, held, lens, free, head, table, slot_capacity, **more)
    ref = _paged.assign(held, lens, list(free), head, table, slot_capacity)
    c.call()
    c.check(ref)
    return c


def start_state(rng, held, max_blocks, spare):
    """A table holding blocks for held tokens, and the free list whose front
    they came from."""
    nb = np.array([blocks_of(max(int(h), 0)) for h in held], np.int64)
    ids = rng.permutation(int(nb.sum()) + spare)
    table = np.full((len(held), max_blocks), -1, np.int64)
    at = 0
    for r, n in enumerate(nb):
        n = min(n, max_blocks)
        table[r, :n] = ids[at:at + n]
        at += n
    return ids, at, table


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,hi,step,cols", [
    (1, 1, 0, 1), (1, 16, 1, 1), (1, 17, 1, 2), (1, 5000, 0, 313),
    (2, 33, 3, 4), (31, 100, 1, 9), (33, 700, 0, 44), (64, 4096, 1, 256),
    (255, 64, 17, 9), (1023, 40, 1, 5), (1025, 90, 0, 6), (4095, 33, 2, 3),
    (4096, 50, 1, 5)])
def test_assign(kv, R, hi, step, cols, in_place):
    rng = np.random.default_rng(R * 1000 + hi)
    lens = rng.integers(0, hi + 1, R)
    lens[0] = hi
    held = np.maximum(lens - step, 0) if step else np.zeros(R, np.int64)
    total = int((lens - held).sum())
    free, head, table = start_state(rng, held, cols, 2 * R + int(
        sum(blocks_of(n) for n in lens)))
    run_assign(kv, held, lens, free, head, table, total + 3,
               in_place=in_place)


def test_assign_large_slot_map(kv):
    # a slot map of more than a million entries, ragged
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 32769, 70)
    lens[3] = lens[40] = 0
    held = np.zeros(70, np.int64)
    free, head, table = start_state(rng, held, 2048, 160000)
    run_assign(kv, held, lens, free, head, table, int(lens.sum()))


@pytest.mark.parametrize("case", range(6))
def test_assign_out_of_the_ordinary(kv, case):
    """Negative and shrinking lengths, requests longer than their table row,
    lists that run out, slot maps too short or absent, ids below zero."""
    rng = np.random.default_rng(case)
    held = np.array([0, -3, 20, 5, 16, 40, 100, 0, 15, 7])
    lens = np.array([30, 4, 10, -1, 32, 41, 120, 65, 17, 7])
    free, head, table = start_state(rng, np.minimum(held, 64), 4, 40)
    cap = 120
    if case == 1:
        free = free[:head + 3]           # room for three more blocks
    elif case == 2:
        cap = 11
    elif case == 3:
        cap = 0
    elif case == 4:
        table[4, 0] = table[8, 0] = -7
        free = free.copy()
        free[head] = -1
    elif case == 5:
        free = free[:0]
        head = 0
    run_assign(kv, held, lens, free, head, table, cap)


@pytest.mark.parametrize("R,cap", [(5, 40), (5, 9000), (1500, 7)])
def test_assign_lengths_far_beyond_the_map(kv, R, cap):
    """Lengths that no table row holds (here near 2^31) cost nothing, and
    blocks are given to tokens that the slot map has no room for."""
    lens = np.full(R, 30)
    lens[1] = 2 ** 31 - 1
    lens[3] = 2 ** 31 - 17
    held = np.zeros(R, np.int64)
    held[3] = 5
    c = Assign(kv, held, lens, np.arange(2 * R), 0, np.full((R, 3), -1), cap)
    c.call()
    table = np.full((R, 3), -1)
    ok = np.ones(R, bool)
    ok[[1, 3]] = False
    table[ok, :2] = np.arange(2 * (R - 2)).reshape(-1, 2)
    np.testing.assert_array_equal(c.table.cpu().numpy(), table)
    np.testing.assert_array_equal(
        c.held_out.cpu().numpy(), np.where(ok, 30, held))
    cu = np.concatenate([[0], np.cumsum(lens - held)])
    np.testing.assert_array_equal(c.cu.cpu().numpy()[:R + 1], cu)
    slots = np.full(cap, -1, np.int64)
    n = min(cap, 30)
    slots[:n] = np.arange(n)          # request 0: blocks 0 and 1
    np.testing.assert_array_equal(c.slots.cpu().numpy()[:cap], slots)
    assert int(c.flags.cpu()[0]) == kv.KVTC_FLAG_SPACE


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,blocks,cap", [
    (1, 40, 0), (7, 300, 0), (64, 33, 0), (1024, 60, 0), (1025, 9, 0),
    (64, 50, 31), (1024, 12, 511), (9, 30, 4)])
def test_assign_of_the_table_alone(kv, R, blocks, cap, in_place):
    """Long prompts with no slot map, or next to none: the table's entries
    are the work, and one block does not write them alone (a state that is
    kept in place is summed in a launch before the one that does)."""
    rng = np.random.default_rng(R + blocks)
    lens = rng.integers(0, 16 * blocks + 1, R)
    lens[R // 2] = 16 * blocks
    held = np.where(rng.random(R) < 0.3, lens // 3, 0)
    free, head, table = start_state(rng, held, blocks, R * blocks)
    n = kv.kvtc_launch_count()
    run_assign(kv, held, lens, free, head, table, cap, in_place=in_place)
    assert kv.kvtc_launch_count() - n == (2 if in_place or R > 1024 else 1)


@pytest.mark.parametrize("R,hi", [(1024, 3), (1025, 3), (4096, 60), (600, 1),
                                  (64, 32), (64, 33), (64, 128), (64, 129)])
def test_assign_with_many_empty_requests(kv, R, hi):
    """Long runs of requests that want nothing, and calls on both sides of
    the 1024 requests of a single launch."""
    rng = np.random.default_rng(R + hi)
    lens = rng.integers(1, hi + 1, R)
    lens[rng.integers(0, R, R // 2)] = 0
    lens[R // 3:R // 3 + R // 4] = 0
    if R == 64:
        lens[:] = hi
    held = np.zeros(R, np.int64)
    free, head, table = start_state(rng, held, blocks_of(hi) + 1,
                                    int(sum(blocks_of(n) for n in lens)) + 5)
    run_assign(kv, held, lens, free, head, table, int(lens.sum()))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("trouble", [None, "list", "map", "table", "ids"])
@pytest.mark.parametrize("R,each", [(7, 15), (7, 17), (64, 16), (64, 18),
                                    (512, 16), (512, 17), (1024, 8),
                                    (1024, 9)])
def test_assign_around_the_limits_of_its_forms(kv, R, each, trouble,
                                               in_place):
    """On both sides of 16 slots a request and of 8192, with the state in
    place and not, where all is well and where something is short."""
    rng = np.random.default_rng(R + each)
    held = rng.integers(0, 20, R)
    lens = held + each
    if trouble == "table":
        lens[R // 2] = 16 * 4 + 1
        held[R // 3] = lens[R // 3] + 3
    free, head, table = start_state(rng, held, 4, 3 * R + 9)
    cap = int(np.maximum(lens - held, 0).sum())
    if trouble == "list":
        free = free[:head + R // 2]
    elif trouble == "map":
        cap = cap // 3
    elif trouble == "ids":
        table[R // 2] = -5
        free = free.copy()
        free[head + 1::7] = -1
    run_assign(kv, held, lens, free, head, table, cap, in_place=in_place)


@pytest.mark.parametrize("head", [-1, 6, 1 << 40])
def test_assign_with_the_head_outside_the_list(kv, head):
    run_assign(kv, [0, 4], [5, 6], [3, 4, 5, 6, 7], head, [[1, 2], [3, 4]],
               9)


def test_assign_without_requests(kv):
    run_assign(kv, np.zeros(0), np.zeros(0), [1, 2], 1, np.zeros((0, 3)), 4)
    run_assign(kv, np.zeros(0), np.zeros(0), [1, 2], 1, np.zeros((0, 3)), 0)


def test_assign_without_a_flag_word(kv):
    c = Assign(kv, [0], [40], [1], 0, [[-1, -1]], 40)
    c.call(flags=False)
    assert int(c.head_out.cpu()[0]) == 0
    assert (c.slots.cpu().numpy()[:40] == -1).all()


def test_assign_steps_replayed_from_a_graph(kv):
    """Decode steps: lengths grow on the device, the state is kept in place,
    and one captured call serves every step."""
    import torch
    rng = np.random.default_rng(11)
    R, cols, steps = 37, 5, 40
    held = rng.integers(0, 30, R)
    free, head, table = start_state(rng, held, cols, 40)
    lens = held.copy()
    c = Assign(kv, held, lens, free, head, table, R + 2, in_place=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    grow = dev(rng.integers(0, 2, R), np.int32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        torch.add(c.held, grow, out=c.lens)
        c.call()
    h, hd, tb = held, head, table
    want = 0
    for i in range(steps):
        new = rng.integers(0, 2, R)
        grow.copy_(dev(new, np.int32))
        g.replay()
        torch.cuda.synchronize()
        tb, slots, cu, h, hd, short = _paged.assign(h, h + new, list(free),
                                                    hd, tb, R + 2)
        want |= c.kv.KVTC_FLAG_SPACE if short else 0
        np.testing.assert_array_equal(c.table.cpu().numpy(), tb)
        np.testing.assert_array_equal(c.slots.cpu().numpy()[:R + 2], slots)
        np.testing.assert_array_equal(c.held.cpu().numpy(), h)
        assert int(c.head.cpu()[0]) == hd
        assert int(c.flags.cpu()[0]) == want


# ------------------------------------------------------------------- append
def append_case(seed, n, width, streams, num_blocks, ld_extra=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = width * streams + ld_extra
    rows = torch.randint(-32768, 32768, (n, ld), generator=g, device="cuda",
                         dtype=torch.int32).to(torch.int16)
    src = [rows[:, j * width:(j + 1) * width] for j in range(streams)]
    cache = [torch.randint(-32768, 32768, (num_blocks, BLOCK, width),
                           generator=g, device="cuda",
                           dtype=torch.int32).to(torch.int16)
             for _ in range(streams)]
    return rows, src, cache, ld


def expect_append(src, cache, slots):
    out = []
    keep = (slots >= 0) & (slots < cache[0].shape[0] * BLOCK)
    for s, c in zip(src, cache):
        x = c.clone().view(-1, c.shape[-1])
        for i in np.nonzero(keep)[0]:
            x[int(slots[i])] = s[int(i)]
        out.append(x.view(c.shape))
    return out


@pytest.mark.parametrize("n,width,streams,ld_extra", [
    (1, 8, 1, 0), (1, 512, 2, 0), (3, 128, 2, 8), (17, 192, 3, 16),
    (64, 512, 2, 1024), (65, 1000, 1, 0), (5, 8192, 2, 0), (300, 1024, 2, 8),
    (7, 64, 65, 0), (2, 72, 130, 0)])
def test_append(kv, n, width, streams, ld_extra):
    import torch
    blocks = blocks_of(n) + 3
    _, src, cache, ld = append_case(n + width, n, width, streams, blocks,
                                    ld_extra)
    slots = np.random.default_rng(n).permutation(blocks * BLOCK)[:n]
    if n > 4:
        slots[[1, n - 1]] = [-1, -(1 << 60)]
    want = expect_append(src, cache, slots)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kvtc_paged_append(src, ld, n, dev(slots, np.int64), width, BLOCK,
                         cache, blocks, flags)
    for a, b in zip(cache, want):
        assert torch.equal(a, b)
    assert int(flags.cpu()[0]) == 0


def test_append_many_rows(kv):
    import torch
    n, width, blocks = 8191, 1024, 600
    _, src, cache, ld = append_case(1, n, width, 2, blocks)
    slots = np.random.default_rng(1).permutation(blocks * BLOCK)[:n]
    at = dev(slots, np.int64)
    want = [c.clone() for c in cache]
    for s, c in zip(src, want):
        c.view(-1, width)[at] = s
    kv.kvtc_paged_append(src, ld, n, at, width, BLOCK, cache, blocks)
    for a, b in zip(cache, want):
        assert torch.equal(a, b)


def test_append_slots_past_the_pool_are_flagged(kv):
    import torch
    n, width, blocks = 9, 64, 2
    _, src, cache, ld = append_case(4, n, width, 2, blocks)
    slots = np.array([31, 32, 5, 1 << 62, 0, -1, 33, 7, 2])
    want = expect_append(src, cache, slots)
    flags = torch.full((1,), 1 << 20, dtype=torch.int32, device="cuda")
    for word in (None, flags):
        kv.kvtc_paged_append(src, ld, n, dev(slots, np.int64), width, BLOCK,
                             cache, blocks, word)
    for a, b in zip(cache, want):
        assert torch.equal(a, b)
    # ORed into what the word held
    assert int(flags.cpu()[0]) == (1 << 20) | kv.KVTC_FLAG_BLOCK


def test_append_into_a_pool_past_32_bits(kv):
    """A pool of more than 2^32 elements: rows at its far end."""
    import torch
    width = 8192
    blocks = (1 << 32) // (BLOCK * width) + 40
    pool = torch.empty((blocks, BLOCK, width), dtype=torch.int16,
                       device="cuda")
    n = 12
    rows = torch.randint(-9999, 9999, (n, width), device="cuda").to(
        torch.int16)
    slots = np.array([0, 5, blocks * BLOCK - 1, (1 << 31) // width,
                      (1 << 32) // width, (1 << 32) // width + 17,
                      blocks * BLOCK - 16, -1, 77, (1 << 18) + 1, 99, 100])
    assert len(set(slots)) == n            # distinct, as the call asks
    pool.view(-1, width)[dev(slots[slots >= 0], np.int64)] = 0
    kv.kvtc_paged_append([rows], width, n, dev(slots, np.int64), width,
                         BLOCK, [pool], blocks)
    for i, s in enumerate(slots):
        if s >= 0:
            assert torch.equal(pool.view(-1, width)[int(s)], rows[i]), i


def test_append_on_another_stream_and_from_a_graph(kv):
    import torch
    n, width, blocks = 33, 256, 4
    _, src, cache, ld = append_case(8, n, width, 2, blocks)
    rng = np.random.default_rng(3)
    at = dev(rng.permutation(blocks * BLOCK)[:n], np.int64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        kv.kvtc_paged_append(src, ld, n, at, width, BLOCK, cache, blocks)
    for _ in range(3):
        slots = rng.permutation(blocks * BLOCK)[:n]
        slots[rng.integers(0, n)] = -1
        at.copy_(dev(slots, np.int64))
        want = expect_append(src, cache, slots)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(cache, want):
            assert torch.equal(a, b)
    want = expect_append(src, cache, at.cpu().numpy())
    st.wait_stream(torch.cuda.current_stream())
    kv.kvtc_paged_append(src, ld, n, at, width, BLOCK, cache, blocks,
                         stream=st)
    st.synchronize()
    for a, b in zip(cache, want):
        assert torch.equal(a, b)


def test_a_missing_device_is_an_error(kv):
    _, src, cache, ld = append_case(8, 2, 64, 1, 2)
    at = dev([0, 1], np.int64)
    with pytest.raises(kv.KvtcError) as e:
        kv.kvtc_paged_append(src, ld, 2, at, 64, BLOCK, cache, 2, device=63,
                             stream=0)
    assert e.value.code == kv.KVTC_ECUDA
    # and the next call works
    kv.kvtc_paged_append(src, ld, 2, at, 64, BLOCK, cache, 2)
    import torch
    assert torch.equal(cache[0].view(-1, 64)[:2], src[0])
