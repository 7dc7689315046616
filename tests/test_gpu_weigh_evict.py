"""Attention weight per cached token, and eviction by it, on the GPU against
the plain forms in 64 bits (needs a GB300)."""
import numpy as np
import pytest

import _chunks
from _paged import BLOCK, bits7, blocks_of, paged_case, softmax_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


class Weigh:
    """Device buffers of one kvtc_paged_weigh call."""

    def __init__(self, kv, seed, news, lens, heads, kv_heads, hd,
                 dtype="bf16", sink=0, window=0, decay=1.0, behind=2,
                 case=None, in_place=False):
        import torch
        t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        self.kv, self.dtype = kv, dtype
        self.heads, self.kv_heads, self.hd = heads, kv_heads, hd
        self.sink, self.window, self.decay = sink, window, decay
        self.scale = softmax_scale(hd)
        _, self.k, _, self.table, self.lens = (
            case or paged_case(seed, lens, heads, kv_heads, hd))
        self.cu = np.concatenate([[0], np.cumsum(news)])
        self.N, self.R = int(self.cu[-1]) + behind, len(lens)
        rng = np.random.default_rng(seed + 1)
        self.q = bits7(rng.standard_normal((self.N, heads, hd)))
        self.width = heads * hd
        # the log-sum-exp of the rows' scores, whatever their values
        self.lse = np.full((self.N, heads), np.nan)
        v = np.zeros_like(self.k)
        with np.errstate(all="ignore"):
            ref = _chunks.attend_chunks(self.q, np.nan_to_num(self.k), v,
                                        self.table, self.cu, self.lens, sink,
                                        window, self.scale, 0.0)
        self.lse[ref[4]] = ref[1][ref[4]]
        self.lse = self.lse.astype(np.float32)
        self.ld = self.table.shape[1] * BLOCK + 4
        self.acc = rng.random((self.R, self.ld)).astype(np.float32)
        self.d_q = torch.full((self.N, self.width + 8), float("nan"),
                              dtype=t, device="cuda")
        self.d_k = torch.from_numpy(self.k).cuda().to(t)
        self.d_acc = torch.zeros((self.R, self.ld), device="cuda")
        self.d_out = self.d_acc if in_place else torch.full_like(self.d_acc,
                                                                 77.0)
        self.in_place = in_place
        self.upload()
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = kv.kvtc_paged_weigh_workspace_bytes(self.R, self.N, heads,
                                                   kv_heads, hd)
        self.ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def upload(self):
        import torch
        self.d_q[:, :self.width].copy_(torch.from_numpy(
            self.q.reshape(self.N, self.width)))
        self.d_lse = torch.from_numpy(self.lse.copy()).cuda()
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_lens = torch.from_numpy(np.array(self.lens, np.int32)).cuda()
        self.d_cu = torch.from_numpy(np.array(self.cu, np.int64)).cuda()
        self.d_acc.copy_(torch.from_numpy(self.acc))

    def call(self, stream=None):
        self.kv.kvtc_paged_weigh(
            self.R, self.N, self.heads, self.kv_heads, self.hd,
            {"bf16": 0, "fp16": 1}[self.dtype], self.d_q,
            self.d_q.stride(0), self.d_k, self.d_k.shape[0], BLOCK,
            self.d_table, self.d_table.shape[1], self.d_cu, self.d_lens,
            self.sink, self.window, self.scale, self.d_lse, self.decay,
            self.d_acc if self.decay else None, self.d_out, self.ld, self.ws,
            self.ws.numel(), self.flags, stream=stream)

    def check(self, flags=0):
        ref, tol = _chunks.weigh(self.q, self.k, self.table, self.cu,
                                 self.lens, self.sink, self.window,
                                 self.scale, self.lse, self.decay, self.acc)
        got = self.d_out.double().cpu().numpy()
        for r, n in enumerate(self.lens):
            n = min(max(int(n), 0), self.table.shape[1] * BLOCK)
            rest = self.acc[r, n:] if self.in_place else 77
            assert (got[r, n:] == rest).all()
            x, y, e = got[r, :n], ref[r, :n], tol[r, :n]
            np.testing.assert_array_equal(np.isnan(x), np.isnan(y))
            far = np.abs(x - y) - e
            far = far[~np.isnan(y)]
            assert far.size == 0 or far.max() <= 0, (r, far.max())
        assert int(self.flags.cpu()[0]) == flags


def weigh(kv, *args, **more):
    a = Weigh(kv, *args, **more)
    a.call()
    a.check()
    return a


NEWS = [0, 1, 2, 15, 16, 17, 31, 33, 5, 0, 1, 64, 100]
LENS = [0, 1, 2, 15, 40, 17, 32, 300, 129, 50, 128, 64, 257]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,hd", [
    (2, 2, 64), (3, 1, 64), (40, 5, 64), (1, 1, 128), (6, 3, 128),
    (32, 8, 128), (28, 4, 128), (66, 2, 128), (9, 9, 128), (2, 2, 256),
    (36, 2, 256), (48, 16, 64)])
def test_weigh_head_layouts(kv, heads, kv_heads, hd, dtype):
    weigh(kv, heads + hd, NEWS, LENS, heads, kv_heads, hd, dtype)


@pytest.mark.parametrize("heads,kv_heads,hd", [
    (1, 1, 64), (28, 4, 128), (8, 8, 128), (32, 2, 128), (12, 3, 256),
    (128, 1, 64), (64, 64, 128)])
def test_weigh_single_tokens(kv, heads, kv_heads, hd):
    lens = [1, 16, 17, 100, 0, 129, 1000]
    news = [1, 1, 1, 1, 0, 1, 1]
    weigh(kv, hd, news, lens, heads, kv_heads, hd)
    weigh(kv, hd, news, lens, heads, kv_heads, hd, "fp16", decay=0.0)


@pytest.mark.parametrize("rows", [1, 2, 7, 32, 65, 128, 300])
def test_weigh_rows(kv, rows):
    weigh(kv, rows, [rows, 1], [rows + 500, 3000], 8, 2, 128)


@pytest.mark.parametrize("R", [33, 200, 4096])
def test_weigh_numbers_of_requests(kv, R):
    rng = np.random.default_rng(R)
    news = rng.integers(0, 3, R)
    weigh(kv, R, news, news + rng.integers(0, 30, R), 2, 1, 64)


@pytest.mark.parametrize("decay", [0.0, 1.0, 0.9, -0.5])
@pytest.mark.parametrize("in_place", [False, True])
def test_weigh_decay(kv, decay, in_place):
    a = weigh(kv, 3, [1, 20], [300, 90], 8, 2, 128, decay=decay,
              in_place=in_place)
    if decay == 0:
        # what acc holds is not read
        b = Weigh(kv, 3, [1, 20], [300, 90], 8, 2, 128, decay=decay)
        b.d_acc.fill_(float("nan"))
        b.call()
        b.check()
    assert a.decay == decay


@pytest.mark.parametrize("sink,window", [(0, 1), (0, 17), (4, 128), (5, 3),
                                         (300, 10), (0, 2147483647),
                                         (2147483647, 1)])
def test_weigh_sink_and_window(kv, sink, window):
    news = [1, 2, 40, 0, 200, 100, 1]
    lens = [1, 18, 40, 30, 300, 1000, 2049]
    case = paged_case(sink % 1000 + window % 1000, lens, 6, 2, 128)
    _, k, v, table, _ = case
    for r, (n, m) in enumerate(zip(lens, news)):
        seen = _chunks.seen_by(n - m + np.arange(m), n, sink, window).any(0)
        t = np.nonzero(~seen)[0]
        k[table[r, t // BLOCK], t % BLOCK] = np.nan
        gone = np.setdiff1d(np.arange(-(-n // BLOCK)),
                            np.nonzero(seen)[0] // BLOCK)
        table[r, gone] = -5
    weigh(kv, 3, news, lens, 6, 2, 128, sink=sink, window=window, case=case)


def test_weigh_without_rows(kv):
    """No rows at all: the sums decay."""
    import torch
    acc = torch.rand((3, 64), device="cuda")
    out = torch.full_like(acc, 77.0)
    lens = torch.tensor([0, 5, 64], dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    cu = torch.zeros(4, dtype=torch.int64, device="cuda")
    pool = torch.zeros((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kv.kvtc_paged_weigh_workspace_bytes(3, 0, 8, 2, 64),
                     dtype=torch.uint8, device="cuda")
    kv.kvtc_paged_weigh(3, 0, 8, 2, 64, 0, None, 512, pool, 1, BLOCK, table,
                        4, cu, lens, 0, 0, 0.125, None, 0.5, acc, out, 64,
                        ws, ws.numel())
    for r, n in enumerate((0, 5, 64)):
        assert torch.equal(out[r, :n], acc[r, :n] * 0.5)
        assert (out[r, n:] == 77).all()


def test_weigh_odd_values(kv):
    lens = [60, 60, 60]
    case = paged_case(5, lens, 4, 2, 64)
    _, k, _, table, _ = case
    k[table[0, 2], 3, 5] = np.nan            # one token, KV head 0
    k[table[1, 1], 0, 64] = -np.inf          # a weight of zero
    a = Weigh(kv, 5, [3, 3, 3], lens, 4, 2, 64, case=case)
    a.q[:, :, 0] = 1.0
    a.lse[a.cu[2] + 1, 2] = -np.inf          # a head that attends to nothing
    a.lse[a.cu[1], 0] = np.nan
    a.upload()
    a.call()
    a.check()


def test_weigh_bad_ids_and_lengths(kv):
    lens = [60, 40, 20]
    case = paged_case(6, lens, 4, 2, 64)
    case[3][0, 1] = -1
    case[3][1, 0] = 10 ** 9
    a = Weigh(kv, 6, [3, 1, 1], lens, 4, 2, 64, case=case)
    a.call()
    a.check(flags=kv.KVTC_FLAG_BLOCK)
    case = paged_case(6, lens, 4, 2, 64, extra_cols=0)
    case[3][2, 2:] = case[3][2, 1]
    a = Weigh(kv, 6, [3, 1, 1], lens, 4, 2, 64, case=case)
    a.lens = np.array([60, -3, 20])
    a.upload()
    a.call()
    a.check()
    a = Weigh(kv, 6, [3, 1, 1], lens, 4, 2, 64, case=case)
    a.lens = np.array([10 ** 6, 40, 20])
    a.k[a.table[0, 3], 12:] = 0.25
    a.d_k.copy_(__import__("torch").from_numpy(a.k))
    a.upload()
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)


def test_weigh_equal_bits_and_graph(kv):
    import torch
    a = weigh(kv, 7, [1, 40, 3], [3000, 700, 9], 28, 4, 128)
    first = a.d_out.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.call()
    for _ in range(3):
        g.replay()
        assert torch.equal(a.d_out, first)
    a.lens = np.array([2000, 650, 9])
    a.d_lens.copy_(torch.from_numpy(a.lens.astype(np.int32)))
    a.d_out.fill_(77)
    g.replay()
    a.check()


@pytest.mark.parametrize("last", [64, 61])
def test_weigh_the_widest_table(kv, last):
    """A request of about 2^31 tokens: its first and last blocks receive what
    those of a short one do, the tokens between them decay."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a = Weigh(kv, 8, [20, 3], [last, 50], 4, 2, 64, sink=3, window=20,
              decay=0.5)
    ref, tol = _chunks.weigh(a.q, a.k, a.table, a.cu, a.lens, a.sink,
                             a.window, a.scale, a.lse, a.decay, a.acc)
    cols = 2 ** 27 - 2
    end = BLOCK * cols                       # of the last block
    n = end - 64 + last
    wide = torch.zeros((2, cols), dtype=torch.int32, device="cuda")
    wide[0, 0] = a.d_table[0, 0]
    wide[0, cols - 3:] = a.d_table[0, 1:4]
    wide[1, :5] = a.d_table[1, :5]
    a.d_table, a.ld = wide, end
    acc = torch.full((2, end), 0.75, device="cuda")
    acc[0, :16] = a.d_acc[0, :16]
    acc[0, end - 48:] = a.d_acc[0, 16:64]
    acc[1, :50] = a.d_acc[1, :50]
    behind = acc[0, n:].clone()
    a.d_acc = a.d_out = acc
    a.d_lens.copy_(torch.tensor([n, 50]))
    a.call()
    torch.cuda.synchronize()
    assert int(a.flags) == 0
    got = torch.cat([acc[0, :16], acc[0, end - 48:n]]).double().cpu().numpy()
    assert (np.abs(got - ref[0, :last]) <= tol[0, :last]).all()
    got = acc[1, :50].double().cpu().numpy()
    assert (np.abs(got - ref[1, :50]) <= tol[1, :50]).all()
    for at in range(16, end - 48, 1 << 28):
        assert (acc[0, at:min(at + (1 << 28), end - 48)] == 0.375).all()
    assert torch.equal(acc[0, n:], behind) and (acc[1, 50:4096] == 0.75).all()


# ------------------------------------------------------------------ evict
class Evict:
    def __init__(self, kv, seed, lens, keep, sink, window, D=64, streams=2,
                 in_place=False, weights=None, cols=None):
        import torch
        rng = np.random.default_rng(seed)
        self.kv, self.keep, self.sink, self.window = kv, keep, sink, window
        self.lens, self.D, self.in_place = np.array(lens), D, in_place
        self.R = len(lens)
        held = np.maximum(self.lens, 0)
        cols = cols or max(1, blocks_of(int(held.max(initial=0)))) + 1
        nb = np.array([blocks_of(int(n)) for n in held])
        kept = np.array([blocks_of(min(int(n), keep)) for n in held])
        total = int(nb.sum() + kept.sum()) + 3
        self.num_blocks = total
        ids = rng.permutation(total)
        self.table = np.full((self.R, cols), 2 ** 31 - 1, np.int32)
        self.out_table = self.table.copy()
        at = 0
        for r in range(self.R):
            self.table[r, :nb[r]] = ids[at:at + nb[r]]
            at += nb[r]
        for r in range(self.R):
            self.out_table[r, :kept[r]] = ids[at:at + kept[r]]
            at += kept[r]
        self.ld = cols * BLOCK
        self.acc = (rng.exponential(size=(self.R, self.ld)) if weights is None
                    else weights(rng, (self.R, self.ld))).astype(np.float32)
        self.pools = [rng.integers(-30000, 30000, (total, BLOCK, D)).astype(
            np.int16) for _ in range(streams)]
        cuda = dict(device="cuda")
        self.d_pools = [torch.from_numpy(p.copy()).cuda() for p in self.pools]
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_out_table = (self.d_table if in_place else
                            torch.from_numpy(self.out_table.copy()).cuda())
        self.d_acc = torch.from_numpy(self.acc.copy()).cuda()
        self.d_acc_out = (self.d_acc if in_place else
                          torch.full_like(self.d_acc, 77.0))
        self.d_lens = torch.from_numpy(self.lens.astype(np.int32)).cuda()
        self.d_lens_out = (self.d_lens if in_place else
                           torch.full_like(self.d_lens, -7))
        self.d_kept = torch.full((self.R + 1, max(keep, 1)), 55,
                                 dtype=torch.int32, **cuda)
        self.flags = torch.zeros(1, dtype=torch.int32, **cuda)
        size = kv.kvtc_paged_evict_workspace_bytes(self.R, cols)
        self.ws = torch.full((size,), 255, dtype=torch.uint8, **cuda)

    def call(self, stream=None):
        self.kv.kvtc_paged_evict(
            self.R, self.d_acc, self.ld, self.d_lens, self.keep, self.sink,
            self.window, self.d_table, self.d_out_table,
            self.table.shape[1], BLOCK, self.d_pools, self.D,
            self.num_blocks,
            self.d_kept if self.keep else None, self.d_acc_out,
            self.d_lens_out, self.ws, self.ws.numel(), self.flags,
            stream=stream)

    def check(self, flags=0):
        start = self.acc if self.in_place else np.full_like(self.acc, 77.0)
        kept, acc, after, pools, _ = _chunks.evict(
            self.acc, self.lens, self.keep, self.sink, self.window,
            self.table, self.table if self.in_place else self.out_table,
            self.pools, self.in_place)
        for r, n in enumerate(self.lens):
            n = min(max(int(n), 0), self.ld)
            acc[r, n:] = start[r, n:]
        got = self.d_kept.cpu().numpy()
        np.testing.assert_array_equal(got[:self.R, :self.keep],
                                      kept[:, :self.keep])
        assert (got[self.R] == 55).all()
        np.testing.assert_array_equal(self.d_lens_out.cpu().numpy(), after)
        np.testing.assert_array_equal(self.d_acc_out.cpu().numpy(), acc)
        for p, x in zip(self.d_pools, pools):
            np.testing.assert_array_equal(p.cpu().numpy(), x)
        assert int(self.flags.cpu()[0]) == flags


LENGTHS = [0, 1, 30, 31, 32, 33, 100, 1023, 1024, 1025, 2500, 5000]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,sink,window", [
    (32, 4, 8), (32, 0, 0), (32, 32, 0), (32, 0, 32), (32, 10, 22),
    (1, 0, 1), (1, 0, 0), (0, 0, 0), (1000, 4, 128), (2000, 0, 1),
    (10 ** 6, 4, 4), (100, 3, 90)])
def test_evict(kv, keep, sink, window, in_place):
    a = Evict(kv, keep + sink, LENGTHS, keep, sink, window,
              in_place=in_place)
    a.call()
    a.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,streams", [(8, 1), (40, 3), (64, 0), (72, 2),
                                       (512, 2), (1024, 65), (8192, 1)])
def test_evict_pools(kv, D, streams, in_place):
    a = Evict(kv, D, [200, 70, 3], 64, 2, 9, D=D, streams=streams,
              in_place=in_place)
    a.call()
    a.check()


def ties(rng, shape):
    return rng.integers(0, 4, shape)


def equal(rng, shape):
    return np.zeros(shape)


def odd(rng, shape):
    x = rng.standard_normal(shape)
    pick = rng.integers(0, 12, shape)
    for i, y in enumerate([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45,
                           -1e-45, 3.4e38]):
        x[pick == i] = y
    x[pick == 8] = np.copysign(np.nan, -1.0)
    return x


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("weights", [ties, equal, odd])
def test_evict_ties_and_odd_weights(kv, weights, in_place):
    for keep in (40, 700):
        a = Evict(kv, keep, [39, 41, 500, 3001], keep, 3, 5, weights=weights,
                  in_place=in_place)
        a.call()
        a.check()


@pytest.mark.parametrize("R", [1, 2, 19, 76, 77, 152, 153, 1000])
def test_evict_numbers_of_requests(kv, R):
    rng = np.random.default_rng(R)
    for in_place in (False, True):
        a = Evict(kv, R, rng.integers(0, 300, R), 100, 4, 16, D=32,
                  in_place=in_place)
        a.call()
        a.check()


@pytest.mark.parametrize("n,keep", [(40000, 5000), (70001, 66000),
                                    (131072, 64)])
def test_evict_long(kv, n, keep):
    for in_place in (False, True):
        a = Evict(kv, n, [n, 50, n // 2], keep, 4, 32, D=16, streams=1,
                  in_place=in_place)
        a.call()
        a.check()


def test_evict_bad_ids_and_lengths(kv):
    for in_place in (False, True):
        a = Evict(kv, 9, [100, 90], 48, 4, 8, in_place=in_place)
        a.table[0, 0] = -1
        a.d_table.copy_(__import__("torch").from_numpy(a.table))
        if not in_place:
            a.out_table[1, 2] = 10 ** 8
            a.d_out_table.copy_(__import__("torch").from_numpy(a.out_table))
        a.call()
        a.check(flags=kv.KVTC_FLAG_BLOCK)
    a = Evict(kv, 10, [96, 90, -4], 48, 4, 8, cols=6)
    a.lens = np.array([10 ** 9, 90, -4])
    a.d_lens.copy_(__import__("torch").from_numpy(a.lens))
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)


def test_evict_graph_and_stream(kv):
    import torch
    a = Evict(kv, 11, [100, 900, 40], 64, 4, 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.call()
    for lens in ([100, 900, 40], [64, 65, 17], [3, 800, 0]):
        a.lens = np.array(lens)
        a.d_lens.copy_(torch.from_numpy(a.lens.astype(np.int32)))
        a.d_acc_out.fill_(77)
        for p, x in zip(a.d_pools, a.pools):
            p.copy_(torch.from_numpy(x))
        g.replay()
        a.check()
    b = Evict(kv, 12, [100, 900, 40], 64, 4, 8, in_place=True)
    st.wait_stream(torch.cuda.current_stream())
    b.call(stream=st)
    st.synchronize()
    b.check()


def test_evict_twice_in_place(kv):
    """What a second cut sees is what the first one left."""
    import torch
    a = Evict(kv, 13, [700, 300], 256, 4, 16, in_place=True)
    a.call()
    a.check()
    b = Evict(kv, 13, [700, 300], 256, 4, 16, in_place=True)
    b.call()
    b.acc = b.d_acc.cpu().numpy().copy()
    b.lens = b.d_lens.cpu().numpy().copy()
    b.pools = [p.cpu().numpy().copy() for p in b.d_pools]
    b.keep = 100
    b.d_kept = torch.full((3, 100), 55, dtype=torch.int32, device="cuda")
    b.call()
    b.check()


@pytest.mark.parametrize("short", [0, 100, 4000])
def test_evict_the_widest_table(kv, short):
    """A request of up to 2^31 - 32 tokens, whose columns share one block but
    for those of the tokens that stay."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    cols, sink, window, D = 2 ** 27 - 2, 3, 40, 16
    n = cols * BLOCK - short
    rng = np.random.default_rng(short)
    # weights below 1 but for 300 heavier ones, and 50 of exactly 1, of which
    # the first 20 stay; around the ends of the blocks' stretches and of the
    # widest 32-bit numbers
    near = [e for c in range(1, 8) for e in (c * (n // 8) - 9,
                                             c * (n // 8) + 60)]
    near += [sink, n - window - 1, n - 4200, n - 4096]
    some = np.unique(np.concatenate([near, rng.integers(sink, n - window,
                                                        400)]))
    some = np.sort(rng.permutation(some)[:350])
    same = np.sort(rng.permutation(350)[:50])
    heavy = np.delete(some, same)
    keep = sink + window + 300 + 20
    kept = np.sort(np.concatenate([np.arange(sink), heavy, some[same][:20],
                                   np.arange(n - window, n)]))
    acc = torch.empty(cols * BLOCK, device="cuda").uniform_(0, 0.999)
    weight = 2 + rng.random(300).astype(np.float32)
    acc[torch.from_numpy(heavy).cuda()] = torch.from_numpy(weight).cuda()
    acc[torch.from_numpy(some[same]).cuda()] = 1.0
    # token t in column t / 16; the columns of the tokens that stay have
    # blocks of their own
    used = np.unique(kept // BLOCK)
    new = blocks_of(keep)
    total = 1 + len(used) + new
    table = torch.zeros(cols, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(used).cuda()] = torch.arange(
        1, 1 + len(used), dtype=torch.int32, device="cuda")
    out_table = torch.full_like(table, -1)
    out_table[:new] = torch.arange(total - new, total, dtype=torch.int32,
                                   device="cuda")
    pool = rng.integers(-30000, 30000, (total, BLOCK, D)).astype(np.int16)
    d_pool = torch.from_numpy(pool).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    d_kept = torch.full((1, keep), 55, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kvtc_paged_evict_workspace_bytes(1, cols),
                     dtype=torch.uint8, device="cuda")
    moved = acc[torch.from_numpy(kept).cuda()]
    tail = acc[n:].clone()
    kv.kvtc_paged_evict(1, acc, cols * BLOCK, lens, keep, sink, window, table,
                        out_table, cols, BLOCK, [d_pool], D, total, d_kept,
                        acc, lens, ws, ws.numel(), flags)
    torch.cuda.synchronize()
    assert int(flags) == 0 and int(lens) == keep
    np.testing.assert_array_equal(d_kept[0].cpu().numpy(), kept)
    assert torch.equal(acc[:keep], moved)
    for a in range(keep, n, 1 << 28):
        assert not acc[a:min(a + (1 << 28), n)].any()
    assert torch.equal(acc[n:], tail)
    j = np.arange(keep)
    pool[total - new + j // BLOCK, j % BLOCK] = pool[
        1 + np.searchsorted(used, kept // BLOCK), kept % BLOCK]
    np.testing.assert_array_equal(d_pool.cpu().numpy(), pool)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("weights", [ties, equal, odd])
@pytest.mark.parametrize("n,R", [(5000, 3), (10000, 3), (20000, 3),
                                 (20000, 20), (20000, 39)])
def test_evict_ties_over_several_blocks(kv, n, R, weights, in_place):
    """Equal and odd weights where two, four and eight blocks choose for a
    request (by the table's width and the number of requests)."""
    for keep in (40, 3000, n - 5):
        lens = [39, n, n // 2 + 7] + [0, 41, 700] * R
        a = Evict(kv, keep + n, lens[:R], keep, 3, 5, D=8, streams=1,
                  weights=weights, in_place=in_place)
        a.call()
        a.check()


def test_weigh_pools_past_32_bits(kv):
    """Blocks past 2^32 elements of the pool."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a = Weigh(kv, 36, [40, 1], [200, 90], 32, 8, 128)
    few = a.k.shape[0]
    blocks = (1 << 32) // (16 * 1024) + few
    wide = torch.zeros((blocks, 16, 1024), dtype=a.d_k.dtype, device="cuda")
    wide[blocks - few:] = a.d_k
    a.d_k = wide
    a.d_table.copy_(torch.where(a.d_table < few, a.d_table + blocks - few,
                                a.d_table))
    a.call()
    a.check()


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_pools_past_32_bits(kv, in_place):
    """Blocks past 2^32 elements of the pools, and others before them."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a = Evict(kv, 14, [200, 70, 3], 64, 2, 9, D=1024, in_place=in_place)
    few = a.num_blocks
    blocks = (1 << 32) // (16 * 1024) + few
    small, wide = a.d_pools, []
    # every second block far away
    at = torch.arange(few, device="cuda")
    at = torch.where(at % 2 == 0, at, at + blocks - few)
    for p in small:
        w = torch.zeros((blocks, 16, 1024), dtype=p.dtype, device="cuda")
        w[at] = p
        wide.append(w)
    for t in {id(x): x for x in (a.d_table, a.d_out_table)}.values():
        t.copy_(torch.where(t < few, at[t.clamp_max(few - 1).long()].int(),
                            t))
    a.d_pools, a.num_blocks = wide, blocks
    a.call()
    a.d_pools = [w[at] for w in wide]
    a.check()
