"""Attention of one new token over paged pools, on the GPU against the plain
form in 64 bits (needs a GB300)."""
import numpy as np
import pytest

import _paged
from _paged import BLOCK, UNIT, blocks_of, check_attend, paged_case, \
    softmax_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


def torch_dtype(dtype):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]


def on_gpu(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(
        torch_dtype(dtype))


class Attend:
    """Device buffers of one kvtc_paged_attend call; q and out are column
    slices of wider rows."""

    def __init__(self, kv, q, k, v, table, lens, dtype="bf16", sink=0,
                 window=0, scale=None, pad=8, lse=True):
        import torch
        self.kv, self.dtype = kv, dtype
        self.R, self.heads, self.hd = q.shape
        self.width = self.heads * self.hd
        self.kv_heads = k.shape[2] // self.hd
        self.num_blocks = k.shape[0]
        self.args = q, k, v, table, lens
        self.sink, self.window = sink, window
        self.scale = softmax_scale(self.hd) if scale is None else scale
        t = torch_dtype(dtype)
        self.q = torch.full((self.R, self.width + pad), float("nan"),
                            dtype=t, device="cuda")
        self.set_q(q)
        self.k, self.v = on_gpu(k, dtype), on_gpu(v, dtype)
        self.table = torch.from_numpy(table.copy()).cuda()
        self.lens = torch.from_numpy(np.array(lens, np.int32)).cuda()
        self.out = torch.full((self.R + 1, self.width + pad), 77.0, dtype=t,
                              device="cuda")
        self.lse = torch.full((self.R + 1, self.heads), 77.0,
                              device="cuda") if lse else None
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = kv.kvtc_paged_attend_workspace_bytes(
            self.R, self.heads, self.kv_heads, self.hd)
        # whatever the workspace holds must not matter: NaN everywhere
        self.ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def set_q(self, q):
        import torch
        self.q[:, :self.width].copy_(
            torch.from_numpy(q.reshape(self.R, self.width)).cuda())

    def call(self, stream=None, ws=None, out=None):
        ws = self.ws if ws is None else ws
        out = self.out if out is None else out
        self.kv.kvtc_paged_attend(
            self.R, self.heads, self.kv_heads, self.hd,
            {"bf16": self.kv.KVTC_DTYPE_BF16,
             "fp16": self.kv.KVTC_DTYPE_FP16}[self.dtype],
            self.q, self.q.stride(0), self.k, self.v, self.num_blocks,
            BLOCK, self.table, self.table.shape[1], self.lens, self.sink,
            self.window, self.scale, out, out.stride(0), self.lse, ws,
            ws.numel(), self.flags, stream=stream)

    def reference(self, q=None, lens=None, table=None):
        q0, k, v, t0, l0 = self.args
        return _paged.attend(q0 if q is None else q, k, v,
                             t0 if table is None else table,
                             l0 if lens is None else lens, self.sink,
                             self.window, self.scale, UNIT[self.dtype])

    def check(self, ref=None, flags=0):
        got = self.out.float().cpu().numpy()
        assert (got[self.R:] == 77).all()
        assert (got[:, self.width:] == 77).all()
        got = got[:self.R, :self.width].reshape(self.R, self.heads, self.hd)
        lse = None
        if self.lse is not None:
            lse = self.lse.double().cpu().numpy()
            assert (lse[self.R:] == 77).all()
            lse = lse[:self.R]
        check_attend(got.astype(np.float64), lse,
                     self.reference() if ref is None else ref)
        assert int(self.flags.cpu()[0]) == flags


def run(kv, seed, lens, heads, kv_heads, hd, dtype="bf16", **more):
    q, k, v, table, lens = paged_case(seed, lens, heads, kv_heads, hd)
    a = Attend(kv, q, k, v, table, lens, dtype, **more)
    a.call()
    a.check()
    return a


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 0, 255, 257]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,hd", [
    (2, 2, 64), (3, 3, 64), (4, 1, 64), (9, 1, 64), (40, 5, 64),
    (1, 1, 128), (6, 3, 128), (32, 8, 128), (28, 4, 128), (64, 8, 128),
    (32, 2, 128), (17, 1, 128), (66, 2, 128), (64, 64, 128),
    (2, 2, 256), (8, 1, 256), (36, 2, 256), (16, 16, 256)])
def test_head_layouts(kv, heads, kv_heads, hd, dtype):
    run(kv, heads + hd, LENS, heads, kv_heads, hd, dtype)


@pytest.mark.parametrize("heads", [2, 3, 5, 8, 15, 16, 24, 31, 33, 64, 100,
                                   127, 128])
def test_group_sizes(kv, heads):
    run(kv, heads, [70, 0, 1, 300], heads, 1, 64)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 127, 128, 129, 1000,
                                    4097, 20011])
def test_one_request(kv, length):
    run(kv, length, [length], 8, 2, 128)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_ragged_batch(kv, hd):
    rng = np.random.default_rng(hd)
    lens = np.concatenate([rng.integers(0, 40, 50), rng.integers(0, 3000, 9),
                           [0, 0, 5001, 1]])
    run(kv, hd, rng.permutation(lens), 12, 4, hd)


def test_many_short_requests(kv):
    rng = np.random.default_rng(4)
    run(kv, 4, rng.integers(0, 20, 4096), 4, 1, 64, "fp16")


@pytest.mark.parametrize("R", [31, 32, 33, 64, 65, 127, 128, 129, 257])
def test_numbers_of_requests(kv, R):
    """On both sides of what a lane and a warp hold of the lengths, empty
    requests, short and long ones mixed."""
    rng = np.random.default_rng(R)
    lens = rng.integers(0, 90, R)
    lens[rng.integers(0, R, R // 4)] = 0
    lens[R // 2] = 700
    lens[-1] = 33
    run(kv, R, lens, 12, 6, 64)


def test_one_request_among_empty_ones(kv):
    lens = np.zeros(700, np.int64)
    lens[311] = 2500
    run(kv, 6, lens, 8, 2, 128)
    run(kv, 7, np.zeros(5, np.int64), 8, 2, 128)


@pytest.mark.parametrize("sink,window", [
    (0, 1), (0, 16), (0, 17), (4, 128), (16, 16), (17, 100), (5, 3),
    (33, 1), (300, 10), (4, 5000), (0, 2147483647), (2147483647, 1)])
def test_sink_and_window(kv, sink, window):
    lens = [0, 1, 5, 16, 18, 40, 131, 132, 133, 145, 300, 1000, 2049]
    q, k, v, table, lens = paged_case(sink + window % 1000, lens, 12, 2, 128)
    # rows outside the window may hold anything
    for r, n in enumerate(lens):
        t = np.setdiff1d(np.arange(n), _paged.attended(n, sink, window))
        k[table[r, t // BLOCK], t % BLOCK] = np.inf
        v[table[r, t // BLOCK], t % BLOCK] = np.nan
        # and blocks wholly outside need no place
        gone = np.setdiff1d(np.arange(blocks_of(n)),
                            _paged.attended(n, sink, window) // BLOCK)
        table[r, gone] = -5
    a = Attend(kv, q, k, v, table, lens, sink=sink, window=window)
    a.call()
    a.check()


@pytest.mark.parametrize("sink,window", [
    (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 1), (0, 2 ** 31 - 1),
    (2 ** 31 - 17, 16)])
@pytest.mark.parametrize("R", [2, 40])
def test_sink_and_window_beyond_every_length(kv, sink, window, R):
    run(kv, 7, [1 + 13 * i for i in range(R)], 8, 4, 64, sink=sink,
        window=window)


def test_the_widest_table(kv):
    """A request of 2^31 - 32 tokens: its first 3 and last 20 are those of a
    short one with the same first and last blocks."""
    import torch
    q, k, v, table, lens = paged_case(8, [64, 64, 50], 16, 2, 64)
    a = Attend(kv, q, k, v, table, lens, sink=3, window=20)
    ref = a.reference()
    cols = 2 ** 27 - 2
    wide = torch.zeros((3, cols), dtype=torch.int32, device="cuda")
    wide[:, 0] = a.table[:, 0]
    wide[:, cols - 2:] = a.table[:, 2:4]
    wide[2] = 0
    wide[2, :4] = a.table[2, :4]
    a.table = wide
    a.lens.copy_(torch.tensor([16 * cols, 16 * cols, 50]))
    a.call()
    a.check(ref)


def test_sink_without_window_is_ignored(kv):
    run(kv, 2, [100, 3], 4, 2, 64, sink=4, window=0)


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0, 1e-30])
def test_scales(kv, scale):
    run(kv, 9, [60, 1, 333], 8, 2, 64, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores(kv, dtype):
    """Scores in the thousands, of both signs: one token takes all weight."""
    q, k, v, table, lens = paged_case(21, [50, 700, 1], 8, 2, 128,
                                      q_scale=300.0)
    a = Attend(kv, q, k, v, table, lens, dtype)
    a.call()
    a.check()


def test_increasing_scores(kv):
    """Each token's score is far above the last one's: the running maximum
    moves at every token."""
    n, hd = 600, 64
    q, k, v, table, lens = paged_case(22, [n, n], 4, 1, hd)
    q[:] = 0
    q[:, :, 0] = 1.0
    for r in range(2):
        t = np.arange(n)
        k[table[r, t // BLOCK], t % BLOCK, 0] = \
            (t if r == 0 else n - t) * 0.25
    a = Attend(kv, q, _paged.bits7(k), v, table, lens, scale=1.0)
    a.call()
    a.check()


def test_infinities_and_nan_in_attended_tokens(kv):
    hd = 64
    q, k, v, table, lens = paged_case(23, [40, 40, 40, 40, 3, 40], 4, 2, hd)
    q[:, :, 0] = 1.0

    def row(pool, r, t, head):
        return pool[table[r, t // BLOCK], t % BLOCK,
                    head * hd:(head + 1) * hd]
    row(k, 0, 20, 0)[0] = -np.inf           # a weight of zero
    row(k, 1, 20, 1)[5] = np.nan            # NaN for KV head 1 alone
    row(v, 2, 39, 0)[7] = np.inf            # an infinite channel
    row(v, 3, 0, 1)[9] = np.nan             # a NaN channel
    for t in range(3):
        row(k, 4, t, 1)[0] = -np.inf        # every weight is zero
    row(k, 5, 33, 0)[0] = np.inf            # s = +inf: inf - inf
    with np.errstate(all="ignore"):
        a = Attend(kv, q, k, v, table, lens)
        a.call()
        ref = a.reference()
    out, lse, tol, tl = ref
    assert np.isnan(out[1, 2:]).all() and np.isfinite(out[1, :2]).all()
    assert (lse[4, 2:] == -np.inf).all() and (out[4, 2:] == 0).all()
    # where the maximum is +inf the formula gives NaN throughout
    out[5, :2] = np.nan
    lse[5, :2] = np.nan
    a.check((out, lse, tol, tl))


def test_bad_block_ids_are_left_out_and_flagged(kv):
    q, k, v, table, lens = paged_case(24, [100, 40, 64, 16], 6, 3, 128)
    clean = table.copy()
    table[0, 2] = -1
    table[2, 3] = k.shape[0]
    table[3, 0] = -2 ** 31                   # nothing is left of it
    a = Attend(kv, q, k, v, table, lens)
    a.call()
    a.check(flags=a.kv.KVTC_FLAG_BLOCK)
    assert (a.out[3, :a.width] == 0).all()
    # the first block of longer requests, and all but the last
    for cut in (slice(0, 1), slice(0, 6)):
        table = clean.copy()
        table[0, cut] = -1
        c = Attend(kv, q, k, v, table, lens)
        c.call()
        c.check(flags=a.kv.KVTC_FLAG_BLOCK)
    # the flag is not set without one
    b = Attend(kv, q, k, v, clean, lens)
    b.call()
    b.check()


def test_lengths_outside_the_table(kv):
    q, k, v, table, lens = paged_case(25, [48, 30, 7], 4, 2, 64,
                                      extra_cols=0)
    table[1, 2] = table[2, 1] = table[2, 2] = 0
    ask = np.array([1000, -9, 7], np.int32)
    a = Attend(kv, q, k, v, table, ask)
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)


def test_requests_that_share_blocks(kv):
    q, k, v, table, lens = paged_case(26, [64, 64, 90], 8, 1, 64)
    table[1, :4] = table[0, :4]
    table[2, :2] = table[0, 1:3]
    a = Attend(kv, q, k, v, table, lens)
    a.call()
    a.check()


@pytest.mark.parametrize("R,heads,kv_heads,hd,longest", [
    (1, 8, 1, 64, 10), (1, 8, 1, 64, 500), (1, 8, 1, 64, 1500),
    (1, 8, 1, 64, 9000), (1, 32, 1, 128, 3000), (1, 16, 1, 256, 700),
    (1, 4, 1, 256, 2500), (5, 7, 1, 128, 3000), (1, 28, 7, 128, 4000),
    (2, 8, 4, 64, 4000), (3, 12, 4, 128, 2000), (1, 15, 15, 64, 2000),
    (9, 16, 4, 128, 900), (12, 6, 6, 64, 600), (38, 40, 1, 128, 300),
    (19, 8, 8, 128, 200), (152, 2, 1, 64, 150), (1, 100, 1, 64, 3000)])
def test_few_items(kv, R, heads, kv_heads, hd, longest):
    """Few requests and KV heads, one of them long and the others short or
    empty: clusters of 1 to 16 blocks to an item."""
    rng = np.random.default_rng(R + longest)
    lens = rng.integers(0, 40, R)
    lens[R // 2] = longest
    if R > 2:
        lens[0] = 0
    run(kv, longest, lens, heads, kv_heads, hd)
    lens[:] = longest - rng.integers(0, min(9, longest), R)
    run(kv, longest + 1, lens[:20], heads, kv_heads, hd, "fp16", sink=3,
        window=longest // 2)


def test_captured_behind_copies_and_other_streams(kv):
    """In a captured graph: behind a memory copy, behind a fill, and behind
    two streams that join."""
    import torch
    q, k, v, table, lens = paged_case(37, [300, 20, 90, 1], 8, 2, 128)
    a = Attend(kv, q, k, v, table, lens)
    # K pool larger than it needs to be, so that the copies take a while
    q_in, k_in = a.q.clone(), a.k.clone()
    lens_in = a.lens.clone()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a.k.copy_(k_in)
        a.out.fill_(77.0)
        a.q.copy_(q_in)
        main.wait_stream(side)
        a.lens.copy_(lens_in)
        a.call()
        a.lens.zero_()
        a.q.zero_()
    for _ in range(3):
        a.k.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        a.check()
        assert (a.lens == 0).all()


def test_launches_are_counted(kv):
    q, k, v, table, lens = paged_case(38, [40], 4, 2, 64)
    a = Attend(kv, q, k, v, table, lens)
    n = kv.kvtc_launch_count()
    a.call()
    assert kv.kvtc_launch_count() - n in (1, 2)


def test_a_missing_device_is_an_error(kv):
    q, k, v, table, lens = paged_case(39, [40], 4, 2, 64)
    a = Attend(kv, q, k, v, table, lens)
    with pytest.raises(kv.KvtcError) as e:
        kv.kvtc_paged_attend(
            1, 4, 2, 64, kv.KVTC_DTYPE_BF16, a.q, a.q.stride(0), a.k, a.v,
            a.num_blocks, BLOCK, a.table, a.table.shape[1], a.lens, 0, 0, 1.0,
            a.out, a.out.stride(0), None, a.ws, a.ws.numel(), device=63,
            stream=0)
    assert e.value.code == kv.KVTC_ECUDA
    a.call()
    a.check()


def test_without_lse(kv):
    run(kv, 27, [33, 0, 900], 8, 2, 64, lse=False)


@pytest.mark.parametrize("pad", [0, 8, 1000])
def test_row_strides(kv, pad):
    run(kv, 28, [33, 0, 200], 6, 2, 128, pad=pad)


def test_pool_past_32_bits(kv):
    """Pools of more than 2^32 elements each, read at their far end."""
    import torch
    hd, heads = 128, 64
    width = heads * hd
    blocks = (1 << 32) // (BLOCK * width) + 9
    q, k, v, table, lens = paged_case(29, [50, 17], heads, heads, hd)
    a = Attend(kv, q, k, v, table, lens)
    small_k, small_v, nb = a.k, a.v, k.shape[0]
    a.k = torch.empty((blocks, BLOCK, width), dtype=small_k.dtype,
                      device="cuda")
    a.v = torch.empty_like(a.k)
    a.k[-nb:], a.v[-nb:] = small_k, small_v
    a.table.copy_(torch.where(a.table < nb, a.table + (blocks - nb),
                              a.table))
    a.num_blocks = blocks
    a.call()
    a.check()


def test_repeated_calls_give_equal_bits(kv):
    a = run(kv, 30, [5000, 3, 812, 0, 64], 28, 4, 128)
    first, lse = a.out.clone(), a.lse.clone()
    for _ in range(5):
        a.out.fill_(77.0)
        a.ws.random_(0, 256)
        a.call()
        import torch
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)


def test_replayed_from_a_graph_with_other_inputs(kv):
    import torch
    q, k, v, table, lens = paged_case(31, [300, 20, 90, 1], 8, 2, 128)
    a = Attend(kv, q, k, v, table, lens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.call()
    rng = np.random.default_rng(0)
    for i in range(4):
        lens2 = np.minimum(lens, rng.integers(0, 301, 4)).astype(np.int32)
        order = rng.permutation(4)
        q2 = _paged.bits7(rng.standard_normal(q.shape))
        a.set_q(q2)
        a.lens.copy_(torch.from_numpy(lens2[order]).cuda())
        a.table.copy_(torch.from_numpy(table[order]).cuda())
        g.replay()
        torch.cuda.synchronize()
        a.check(a.reference(q=q2, lens=lens2[order], table=table[order]))


def test_two_graphs_that_share_a_workspace(kv):
    """Captured apart, replayed in turn on one stream."""
    import torch
    a = run(kv, 32, [700, 2, 90], 8, 2, 128)
    b = run(kv, 33, [40, 1900], 4, 1, 64, "fp16")
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for c in (a, b):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c.call(ws=ws)
        graphs.append(g)
    for c in (a, b):
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_calls_at_once_on_two_streams(kv):
    import torch
    a = run(kv, 34, [3000, 2, 90], 8, 2, 128)
    b = run(kv, 35, [40, 2900], 8, 2, 128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, st in zip((a, b), streams):
        c.out.fill_(77.0)
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, st in zip((a, b), streams):
            c.call(stream=st)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_parts_joined_by_their_lse(kv):
    """A request's blocks split over two rows, the two results joined: the
    whole, within both parts' bounds."""
    q, k, v, table, lens = paged_case(36, [200], 8, 2, 64)
    whole = _paged.attend(q, k, v, table, lens, 0, 0, softmax_scale(64), 0.0)
    split = np.stack([table[0, :13], np.roll(table[0, :13], -5)])
    q2 = np.concatenate([q, q])
    a = Attend(kv, q2, k, v, split, np.array([80, 120], np.int32))
    a.call()
    a.check()
    out = a.out[:2, :a.width].double().cpu().numpy().reshape(2, 8, 64)
    lse = a.lse[:2].double().cpu().numpy()
    both = _paged.log_add(lse[0], lse[1])
    joined = sum(out[i] * np.exp(lse[i] - both)[:, None] for i in range(2))
    # each part's rounding (2^-8 of its value), weighted by its share
    bound = sum(np.abs(out[i]) * np.exp(lse[i] - both)[:, None]
                for i in range(2)) * 2.0 ** -8 + 2e-4
    assert (np.abs(joined - whole[0][0]) <= bound).all()
    np.testing.assert_allclose(both, whole[1][0], rtol=0, atol=1e-4)
