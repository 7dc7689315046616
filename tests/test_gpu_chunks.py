"""Attention of chunks of new tokens over paged pools, on the GPU against the
plain form in 64 bits (needs a GB300)."""
import numpy as np
import pytest

import _chunks
import _paged
from _chunks import check_chunks
from _paged import BLOCK, UNIT, bits7, paged_case, softmax_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


def on_gpu(x, dtype):
    import torch
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(t)


class Chunks:
    """Device buffers of one kvtc_paged_attend_chunks call; q and out are
    column slices of wider rows, with rows of no request before and behind
    (NaN in q)."""

    def __init__(self, kv, seed, news, lens, heads, kv_heads, hd,
                 dtype="bf16", sink=0, window=0, scale=None, before=0,
                 behind=3, lse=True, case=None):
        import torch
        self.kv, self.dtype = kv, dtype
        self.heads, self.kv_heads, self.hd = heads, kv_heads, hd
        self.sink, self.window = sink, window
        self.scale = softmax_scale(hd) if scale is None else scale
        _, self.k, self.v, self.table, self.lens = (
            case or paged_case(seed, lens, heads, kv_heads, hd))
        self.cu = before + np.concatenate([[0], np.cumsum(news)])
        self.N = int(self.cu[-1]) + behind
        self.R, self.width = len(lens), heads * hd
        rng = np.random.default_rng(seed + 1)
        self.q = bits7(rng.standard_normal((self.N, heads, hd)))
        self.q[:before] = np.nan
        self.q[self.N - behind:] = np.nan
        t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        self.d_q = torch.full((self.N, self.width + 8), float("nan"),
                              dtype=t, device="cuda")
        self.out = torch.full((self.N + 1, self.width + 8), 77.0, dtype=t,
                              device="cuda")
        self.lse = torch.full((self.N + 1, heads), 77.0,
                              device="cuda") if lse else None
        self.d_k, self.d_v = on_gpu(self.k, dtype), on_gpu(self.v, dtype)
        self.upload()
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = kv.kvtc_paged_attend_chunks_workspace_bytes(
            self.R, self.N, heads, kv_heads, hd)
        # whatever the workspace holds must not matter: NaN everywhere
        self.ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def upload(self):
        import torch
        self.d_q[:, :self.width].copy_(
            torch.from_numpy(self.q.reshape(self.N, self.width)).cuda())
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_lens = torch.from_numpy(np.array(self.lens, np.int32)).cuda()
        self.d_cu = torch.from_numpy(np.array(self.cu, np.int64)).cuda()

    def call(self, stream=None, ws=None):
        ws = self.ws if ws is None else ws
        self.kv.kvtc_paged_attend_chunks(
            self.R, self.N, self.heads, self.kv_heads, self.hd,
            {"bf16": 0, "fp16": 1}[self.dtype], self.d_q,
            self.d_q.stride(0), self.d_k, self.d_v, self.d_k.shape[0], BLOCK,
            self.d_table, self.d_table.shape[1], self.d_cu, self.d_lens,
            self.sink, self.window, self.scale, self.out,
            self.out.stride(0), self.lse, ws, ws.numel(), self.flags,
            stream=stream)

    def reference(self):
        return _chunks.attend_chunks(self.q, self.k, self.v, self.table,
                                     self.cu, self.lens, self.sink,
                                     self.window, self.scale,
                                     UNIT[self.dtype])

    def check(self, ref=None, flags=0):
        ref = self.reference() if ref is None else ref
        got = self.out.double().cpu().numpy()
        has = ref[4]
        none = np.concatenate([~has, [True]])
        assert (got[none] == 77).all() and (got[:, self.width:] == 77).all()
        got = got[:self.N, :self.width].reshape(self.N, self.heads, self.hd)
        lse = None
        if self.lse is not None:
            lse = self.lse.double().cpu().numpy()
            assert (lse[none] == 77).all()
            lse = lse[:self.N]
        check_chunks(got, lse, ref)
        assert int(self.flags.cpu()[0]) == flags


def run(kv, seed, news, lens, heads, kv_heads, hd, dtype="bf16", **more):
    a = Chunks(kv, seed, news, lens, heads, kv_heads, hd, dtype, **more)
    a.call()
    a.check()
    return a


NEWS = [0, 1, 2, 15, 16, 17, 31, 33, 5, 0, 1, 64, 100]
LENS = [0, 1, 2, 15, 40, 17, 32, 300, 129, 50, 128, 64, 257]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,hd", [
    (2, 2, 64), (3, 1, 64), (40, 5, 64), (1, 1, 128), (6, 3, 128),
    (32, 8, 128), (28, 4, 128), (12, 1, 128), (66, 2, 128), (2, 2, 256),
    (8, 1, 256), (36, 2, 256)])
def test_head_layouts(kv, heads, kv_heads, hd, dtype):
    run(kv, heads + hd, NEWS, LENS, heads, kv_heads, hd, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,hd", [
    (2, 2, 64), (15, 3, 64), (1, 1, 128), (28, 4, 128), (9, 1, 128),
    (2, 2, 256), (24, 2, 256)])
def test_runs_over_a_wide_table(kv, heads, kv_heads, hd, dtype):
    """Under a table of more than 64 columns items are dealt out in runs that
    begin and end inside them, and joined by a second launch."""
    case = paged_case(heads, LENS, heads, kv_heads, hd, extra_cols=70)
    before = kv.kvtc_launch_count()
    a = run(kv, heads, NEWS, LENS, heads, kv_heads, hd, dtype, case=case)
    assert kv.kvtc_launch_count() == before + 2
    # the same call under a narrow one: a block per item
    narrow = paged_case(heads, LENS, heads, kv_heads, hd)
    few = sum(-(-n // max(1, 128 // (heads // kv_heads))) for n in NEWS)
    b = Chunks(kv, heads, NEWS, LENS, heads, kv_heads, hd, dtype,
               case=narrow)
    before = kv.kvtc_launch_count()
    b.call()
    b.check()
    count = kv.kvtc_launch_count() - before
    assert count in (1, 2) and (count == 1 or (few + 13) * kv_heads > 152)
    assert a.R == b.R


@pytest.mark.parametrize("new,held", [(1, 20000), (3, 4000), (200, 3000),
                                      (64, 64000)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_few_rows_over_many_blocks(kv, new, held, hd):
    """One item cut into parts for many blocks, and their join."""
    run(kv, new + hd, [new], [new + held], 2, 1, hd)


@pytest.mark.parametrize("group", [5, 24, 31, 33, 64, 65, 100, 127, 128])
def test_group_sizes(kv, group):
    run(kv, group, [3, 0, 1, 9], [70, 0, 1, 300], group, 1, 64)


@pytest.mark.parametrize("new,held", [
    (1, 0), (1, 5000), (128, 0), (127, 1), (129, 127), (256, 256), (257, 255),
    (513, 3), (1000, 1200), (40, 9000)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_one_request(kv, new, held, hd):
    run(kv, new + hd, [new], [new + held], 4, 2, hd)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_ragged_batch(kv, hd):
    rng = np.random.default_rng(hd)
    news = np.concatenate([np.ones(20, np.int64), rng.integers(0, 40, 20),
                           rng.integers(100, 300, 4)])
    held = np.concatenate([rng.integers(0, 900, 40), rng.integers(0, 50, 4)])
    at = rng.permutation(len(news))
    run(kv, hd, news[at], (news + held)[at], 12, 4, hd, before=5)


def test_many_requests(kv):
    rng = np.random.default_rng(4)
    news = rng.integers(0, 3, 4096)
    run(kv, 4, news, news + rng.integers(0, 12, 4096), 2, 1, 64, "fp16")


@pytest.mark.parametrize("R", [31, 32, 33, 127, 129, 257])
def test_numbers_of_requests(kv, R):
    rng = np.random.default_rng(R)
    news = rng.integers(0, 20, R)
    news[rng.integers(0, R, R // 4)] = 0
    lens = news + rng.integers(0, 60, R)
    news[R // 2] = 90
    lens[R // 2] = 700
    run(kv, R, news, lens, 6, 3, 64)


def test_no_rows_at_all(kv):
    a = run(kv, 7, [0, 0, 0], [5, 0, 100], 4, 2, 64)
    assert (a.out == 77).all()


@pytest.mark.parametrize("sink,window", [
    (0, 1), (0, 16), (0, 17), (4, 128), (16, 16), (17, 100), (5, 3),
    (33, 1), (300, 10), (130, 129), (4, 5000), (0, 2147483647),
    (2147483647, 1), (2147483647, 2147483647)])
def test_sink_and_window(kv, sink, window):
    news = [1, 2, 40, 0, 200, 100, 7, 300]
    lens = [1, 18, 40, 30, 300, 1000, 2049, 300]
    case = paged_case(sink % 1000 + window % 1000, lens, 6, 2, 128)
    _, k, v, table, _ = case
    # tokens that no row attends to may hold anything and need no place
    for r, (n, m) in enumerate(zip(lens, news)):
        seen = _chunks.seen_by(n - m + np.arange(m), n, sink, window).any(0)
        t = np.nonzero(~seen)[0]
        k[table[r, t // BLOCK], t % BLOCK] = np.inf
        v[table[r, t // BLOCK], t % BLOCK] = np.nan
        gone = np.setdiff1d(np.arange(-(-n // BLOCK)),
                            np.nonzero(seen)[0] // BLOCK)
        table[r, gone] = -5
    run(kv, 3, news, lens, 6, 2, 128, sink=sink, window=window, case=case)


def test_the_widest_table(kv):
    """A request of 2^31 - 32 tokens: what its rows attend to is what those
    of a short one with the same first and last blocks do."""
    import torch
    a = Chunks(kv, 8, [20, 3], [64, 50], 4, 2, 64, sink=3, window=20)
    ref = a.reference()
    cols = 2 ** 27 - 2
    wide = torch.zeros((2, cols), dtype=torch.int32, device="cuda")
    wide[0, 0] = a.d_table[0, 0]
    wide[0, cols - 3:] = a.d_table[0, 1:4]
    wide[1, :5] = a.d_table[1, :5]
    a.d_table = wide
    a.d_lens.copy_(torch.tensor([16 * cols, 50]))
    a.call()
    a.check(ref)


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0, 1e-30])
def test_scales(kv, scale):
    run(kv, 9, [30, 1, 140], [60, 1, 333], 8, 2, 64, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores(kv, dtype):
    """Scores in the thousands, of both signs: one token takes all weight."""
    a = Chunks(kv, 21, [50, 20, 1], [50, 700, 1], 8, 2, 128, dtype)
    a.q *= 256.0
    a.upload()
    a.call()
    a.check()


@pytest.mark.parametrize("hd", [64, 256])
def test_increasing_scores(kv, hd):
    """Each token's score is far above (below) the last one's: the running
    maximum moves at every token, or is the first."""
    n, case = 600, None
    case = paged_case(22, [n, n], 4, 1, hd)
    _, k, v, table, _ = case
    for r in range(2):
        t = np.arange(n)
        k[table[r, t // BLOCK], t % BLOCK, 0] = bits7(
            (t if r == 0 else n - t) * 0.25)
    a = Chunks(kv, 1, [400, 300], [n, n], 4, 1, hd, scale=1.0, case=case)
    a.q[:] = 0
    a.q[:, :, 0] = 1.0
    a.upload()
    a.call()
    a.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_infinities_and_nan_reach_who_attends(kv, hd, dtype):
    """Odd values in K, V and q: the rows that attend to them get the
    formula's result, the others are untouched."""
    news, lens = [40, 150, 40, 3, 40, 140], [40, 300, 90, 3, 40, 140]
    case = paged_case(23, lens, 4, 2, hd)
    _, k, v, table, _ = case

    def row(pool, r, t, head):
        return pool[table[r, t // BLOCK], t % BLOCK,
                    head * hd:(head + 1) * hd]
    row(v, 0, 20, 0)[7] = np.inf            # rows 20 on
    row(v, 0, 39, 1)[9] = np.nan            # the last row alone
    row(v, 1, 200, 0)[3] = -np.inf          # rows from the middle on
    row(v, 1, 299, 0)[3] = np.inf           # and the last: inf - inf
    row(k, 2, 70, 1)[5] = np.nan
    for t in range(3):
        row(k, 3, t, 1)[0] = -np.inf        # every weight is zero
    row(k, 4, 33, 0)[0] = -np.inf           # a weight of zero
    a = Chunks(kv, 24, news, lens, 4, 2, hd, dtype, case=case)
    a.q[:, :, 0] = 1.0
    a.q[a.cu[5] + 6, 3, 1] = np.nan         # one row's head
    a.upload()
    a.call()
    with np.errstate(all="ignore"):
        ref = a.reference()
    out, lse = ref[0], ref[1]
    assert np.isfinite(out[a.cu[0]:a.cu[0] + 20]).all()
    assert np.isinf(out[a.cu[0] + 20:a.cu[1], :2, 7]).all()
    assert np.isnan(out[a.cu[2] - 1, 0, 3]) and np.isinf(
        out[a.cu[2] - 2, 0, 3])
    assert (out[a.cu[3]:a.cu[4], 2:] == 0).all()
    a.check(ref)


@pytest.mark.parametrize("sink,window", [(4, 100), (20, 33)])
def test_nan_behind_the_window(kv, sink, window):
    """A NaN in V that the first rows of a chunk attend to and the later ones,
    whose window has moved on, do not; and one in the sink."""
    new, n, hd = 200, 420, 128
    case = paged_case(33, [n], 4, 2, hd)
    _, k, v, table, _ = case
    for t, c in ((n - new - 10, 5), (n - new - window + 3, 6), (2, 9)):
        v[table[0, t // BLOCK], t % BLOCK, c] = np.nan
    a = Chunks(kv, 3, [new], [n], 4, 2, hd, sink=sink, window=window,
               case=case)
    a.call()
    ref = a.reference()
    assert np.isnan(ref[0][:new, :2, 9]).sum() == 2 * new
    assert 0 < np.isnan(ref[0][:new, :2, 5]).sum() < 2 * new
    a.check(ref)


def test_bad_block_ids_are_left_out_and_flagged(kv):
    news, lens = [30, 40, 64, 16], [100, 40, 200, 16]
    case = paged_case(24, lens, 6, 3, 128)
    _, k, v, table, _ = case
    clean = table.copy()
    table[0, 2] = -1
    table[2, 3] = k.shape[0]
    table[3, 0] = -2 ** 31                   # nothing is left of it
    a = run_flagged(kv, news, lens, case, kv.KVTC_FLAG_BLOCK)
    assert (a.out[int(a.cu[3]):int(a.cu[4]), :a.width] == 0).all()
    for cut in (slice(0, 1), slice(0, 6), slice(0, 9)):
        table[:] = clean
        table[2, cut] = -1
        run_flagged(kv, news, lens, case, kv.KVTC_FLAG_BLOCK)
    table[:] = clean
    run_flagged(kv, news, lens, case, 0)


def run_flagged(kv, news, lens, case, flags):
    a = Chunks(kv, 24, news, lens, 6, 3, 128, case=case)
    a.call()
    a.check(flags=flags)
    return a


def test_lengths_outside_the_table(kv):
    case = paged_case(25, [48, 30, 7, 33], 4, 2, 64, extra_cols=0)
    table = case[3]
    table[1, 2] = table[2, 1] = table[2, 2] = 0
    a = Chunks(kv, 2, [20, 5, 9, 33], [48, 30, 7, 33], 4, 2, 64, case=case)
    # above the table; negative; more rows than tokens; whole
    a.lens = np.array([1000, -9, 7, 33])
    a.upload()
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)
    assert (a.out[int(a.cu[1]):int(a.cu[2]), :a.width] == 0).all()
    assert (a.out[int(a.cu[2]):int(a.cu[2]) + 2, :a.width] == 0).all()
    assert (a.lse[int(a.cu[1]):int(a.cu[2])] == -float("inf")).all()


def test_rows_outside(kv):
    """cu beyond N counts as N."""
    a = Chunks(kv, 26, [10, 20], [30, 40], 4, 2, 64, behind=0)
    a.cu = np.array([0, 10, 34])
    a.upload()
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)
    a = Chunks(kv, 26, [10, 20], [30, 40], 4, 2, 64, behind=0)
    a.cu = np.array([-4, 10, 30])
    a.upload()
    a.call()
    a.check()


def test_requests_that_share_blocks(kv):
    case = paged_case(27, [64, 64, 90], 8, 1, 64)
    table = case[3]
    table[1, :4] = table[0, :4]
    table[2, :2] = table[0, 1:3]
    run(kv, 27, [5, 64, 30], [64, 64, 90], 8, 1, 64, case=case)


def test_equal_calls_give_equal_bits(kv):
    import torch
    a = run(kv, 28, [300, 1, 77, 5], [900, 4000, 77, 2500], 16, 4, 128)
    first = a.out.clone(), a.lse.clone()
    for _ in range(3):
        a.ws.fill_(0)
        a.call()
        assert torch.equal(a.out, first[0]) and torch.equal(a.lse, first[1])


def test_without_lse(kv):
    run(kv, 29, [30, 2], [100, 700], 4, 2, 128, lse=False)


def test_graph_replayed_with_other_lengths(kv):
    import torch
    a = Chunks(kv, 30, [40, 100, 7], [500, 100, 300], 8, 2, 128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.call()
    for news, lens in (([40, 100, 7], [500, 100, 300]),
                       ([1, 1, 1], [17, 3, 290]), ([0, 90, 57], [9, 95, 57])):
        a.cu = np.concatenate([[0], np.cumsum(news)])
        a.lens = np.array(lens)
        a.d_cu.copy_(torch.from_numpy(a.cu))
        a.d_lens.copy_(torch.from_numpy(a.lens.astype(np.int32)))
        a.out.fill_(77)
        a.lse.fill_(77)
        a.q = np.where(np.isnan(a.q), 0.5, a.q)
        a.d_q[:, :a.width].copy_(torch.from_numpy(
            a.q.reshape(a.N, a.width)))
        g.replay()
        a.check()


def test_two_streams(kv):
    import torch
    a = Chunks(kv, 31, [200, 1], [800, 3000], 8, 2, 128)
    b = Chunks(kv, 32, [33, 150], [900, 150], 8, 2, 128)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.call(stream=s)
        b.call(stream=t)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_one_workspace_call_after_call(kv):
    import torch
    a = Chunks(kv, 34, [64, 3], [300, 2000], 8, 2, 128)
    b = Chunks(kv, 35, [9, 150], [900, 150], 8, 2, 128)
    ws = torch.full((max(a.ws.numel(), b.ws.numel()),), 255,
                    dtype=torch.uint8, device="cuda")
    for _ in range(3):
        a.call(ws=ws)
        b.call(ws=ws)
    a.check()
    b.check()


def test_pools_past_32_bits(kv):
    """Blocks past 2^32 elements of the pools."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a = Chunks(kv, 36, [40, 1], [200, 90], 32, 8, 128)
    blocks = (1 << 32) // (16 * 1024) + a.k.shape[0]
    far = blocks - a.k.shape[0]
    pools = []
    for p in (a.d_k, a.d_v):
        wide = torch.zeros((blocks, 16, 1024), dtype=p.dtype, device="cuda")
        wide[far:] = p
        pools.append(wide)
    ref = a.reference()
    a.d_k, a.d_v = pools
    has = a.d_table < a.k.shape[0]
    a.d_table.copy_(torch.where(has, a.d_table + far, a.d_table))
    a.call()
    a.check(ref)


def test_joins_with_the_single_token_call(kv):
    """A chunk of one token a request is what kvtc_paged_attend gives."""
    import torch
    lens = [1, 40, 300, 2000]
    a = run(kv, 37, [1] * 4, lens, 8, 2, 128, behind=0)
    out, lse = torch.empty_like(a.out[:4]), torch.empty_like(a.lse[:4])
    ws = torch.empty(kv.kvtc_paged_attend_workspace_bytes(4, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    kv.kvtc_paged_attend(4, 8, 2, 128, 0, a.d_q, a.d_q.stride(0), a.d_k,
                         a.d_v, a.d_k.shape[0], BLOCK, a.d_table,
                         a.d_table.shape[1], a.d_lens, 0, 0, a.scale, out,
                         out.stride(0), lse, ws, ws.numel())
    ref = _paged.attend(a.q, a.k, a.v, a.table, a.lens, 0, 0, a.scale,
                        UNIT["bf16"])
    _paged.check_attend(out[:, :a.width].double().cpu().numpy().reshape(
        4, 8, 128), lse.double().cpu().numpy(), ref)
    # scores off by 2^-21 or so each: the statistics agree far closer than
    # the outputs' rounding
    assert (lse - a.lse[:4]).abs().max() < 1e-4


@pytest.mark.parametrize("heads,kv_heads,hd", [
    (16, 16, 128), (8, 8, 256), (24, 12, 64), (28, 4, 128)])
def test_single_rows_over_scattered_pools(kv, heads, kv_heads, hd):
    """Many single rows over long contexts whose pages lie far apart, so that
    loads land in another order than they were asked for: against the plain
    form, and call after call to the same bits."""
    import torch
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    R, D = 64, kv_heads * hd
    rng = np.random.default_rng(hd + heads)
    lens = rng.permutation(1 + 8191 * np.arange(R) // (R - 1))
    blocks = -(-lens // BLOCK)
    cols, total = int(blocks.max()), (8 << 30) // (2 * BLOCK * D)
    table = np.full((R, cols), -1, np.int32)
    table[np.arange(cols)[None, :] < blocks[:, None]] = rng.permutation(
        total)[:blocks.sum()]
    k, v = (torch.empty((total, BLOCK, D), dtype=torch.bfloat16,
                        device="cuda").normal_() for _ in range(2))
    q = torch.randn((R, heads * hd), device="cuda").bfloat16()
    d_table, d_lens = torch.from_numpy(table).cuda(), torch.from_numpy(
        lens.astype(np.int32)).cuda()
    cu = torch.arange(R + 1, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kvtc_paged_attend_chunks_workspace_bytes(
        R, R, heads, kv_heads, hd), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        other = torch.zeros(4 << 30, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        lse = torch.zeros((R, heads), device="cuda")
        kv.kvtc_paged_attend_chunks(
            R, R, heads, kv_heads, hd, kv.KVTC_DTYPE_BF16, q, q.stride(0), k,
            v, total, BLOCK, d_table, cols, cu, d_lens, 0, 0, hd ** -0.5,
            out, out.stride(0), lse, ws, ws.numel(), flags=flags)
        torch.cuda.synchronize()
        del other
        assert int(flags) == 0
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    group = heads // kv_heads
    for r in range(0, R, 3):
        t = torch.arange(int(lens[r]), device="cuda")
        at = d_table[r].long()[t // BLOCK] * BLOCK + t % BLOCK
        keys = k.view(-1, kv_heads, hd)[at].double()
        vals = v.view(-1, kv_heads, hd)[at].double()
        rows = q[r].double().view(kv_heads, group, hd)
        x = torch.einsum("jgd,tjd->jgt", rows, keys) * hd ** -0.5
        top = torch.logsumexp(x, -1)
        p = torch.exp(x - top[..., None])
        o = torch.einsum("jgt,tjd->jgd", p, vals)
        # weights and outputs rounded to bf16 (2^-8 each); a score is a sum
        # of hd products in fp32, off by less than hd 2^-24 sum |q k| scale,
        # here below 2^-24 hd^1.5 < 2^-12
        most = torch.einsum("jgt,tjd->jgd", p, vals.abs())
        tol = (2.0 ** -8 + 2.0 ** -11) * most + 2.0 ** -8 * o.abs() * 1.01
        off = (out[r].double().view(kv_heads, group, hd) - o).abs()
        assert (off <= tol).all(), (r, float((off - tol).max()))
        assert (lse[r].double().view(kv_heads, group) - top).abs().max() < (
            2.0 ** -11)


@pytest.mark.parametrize("mean,most", [(0.0, 1.5), (2.0, 1.1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_error_beside_the_output_rounding(kv, dtype, mean, most):
    """The error against 64 bits in the 2-norm, over that of rounding the
    64-bit result once.  A weight's rounding to 16 bits is as large, relative,
    as the output's.  Where V has no mean, so that its products cancel as they
    add up, the two count alike: sqrt(2), to a few percent by where in a binade
    the outputs lie.  Where V's mean is twice its spread, the weights' errors
    cancel instead: against the output they fall by the root of the number of
    tokens."""
    import torch
    new, n = 200, 1900
    case = paged_case(41, [n], 4, 2, 128)
    _, _, v, table, _ = case
    t = np.arange(n)
    rng = np.random.default_rng(42)
    v[table[0, t // BLOCK], t % BLOCK] = bits7(
        rng.standard_normal((n, v.shape[2])) + mean)
    a = Chunks(kv, 43, [new], [n], 4, 2, 128, dtype, case=case)
    a.call()
    ref = a.reference()
    a.check(ref)
    exact = torch.from_numpy(ref[0][:new])
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    once = float((exact.to(t).double() - exact).norm())
    off = float((a.out[:new, :a.width].cpu().double().view(exact.shape) -
                 exact).norm())
    assert off <= most * once


@pytest.mark.parametrize("heads,kv_heads,hd,news,cols,launches", [
    (2, 2, 64, [16], 16, 1), (2, 2, 64, [16], 64, 1),
    (2, 2, 64, [16], 65, 2),
    # 18 tokens of 7 heads to a tile, two tiles an item (one at head_dim 256):
    # 4 (12 + 26) items, and one request more
    (28, 4, 128, [16] * 26, 8, 1), (28, 4, 128, [16] * 26 + [0], 8, 2),
    (1, 1, 256, [128] * 76, 8, 1), (1, 1, 256, [128] * 76 + [1], 8, 2),
    (1, 1, 64, [256] * 76, 16, 1), (1, 1, 64, [256] * 76 + [1], 16, 2)])
def test_launches_by_items_and_columns(kv, heads, kv_heads, hd, news, cols,
                                       launches):
    """One launch where the table has at most 64 columns and there are at most
    as many items, kv_heads (ceil(N / rows of an item) + R), as SMs."""
    rows = 128 // (heads // kv_heads) * (1 if hd == 256 else 2)
    items = kv_heads * (-(-sum(news) // rows) + len(news))
    assert launches == (1 if items <= 152 and cols <= 64 else 2)
    most = -(-max(news) // BLOCK)
    case = paged_case(5, news, heads, kv_heads, hd, extra_cols=cols - most)
    a = Chunks(kv, 6, news, news, heads, kv_heads, hd, case=case, behind=0)
    assert a.d_table.shape[1] == cols
    before = kv.kvtc_launch_count()
    a.call()
    assert kv.kvtc_launch_count() - before == launches
    a.check()


@pytest.mark.parametrize("news,lens,launches", [
    ([16], 500, 1), ([16], 512, 1), ([16], 528, 2), ([16], 1000, 2),
    # 75, 77 and 153 items
    ([1] * 74, 1000, 2), ([1] * 76, 1000, 1), ([1] * 152, 300, 2)])
def test_launches_at_head_dim_256(kv, news, lens, launches):
    """A block takes units of 64 tokens there: one launch up to 32 columns, up
    to 64 where more than 76 items keep the SMs busy."""
    lens = [lens] + [40] * (len(news) - 1)
    case = paged_case(7, lens, 1, 1, 256, extra_cols=0)
    a = Chunks(kv, 8, news, lens, 1, 1, 256, case=case, behind=0)
    before = kv.kvtc_launch_count()
    a.call()
    assert kv.kvtc_launch_count() - before == launches
    a.check()
