"""Norms and rotation of new tokens' rows into the pools, on the GPU against
the plain form in 64 bits (needs a GB300)."""
import numpy as np
import pytest

import _chunks
from _paged import BLOCK, UNIT, bits7

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


class Rotate:
    """Device buffers of one kvtc_paged_rotate call: q, k and v are slices of
    wider rows, pools and q_out hold 77 where nothing is written."""

    def __init__(self, kv, N, heads, kv_heads, hd, dtype="bf16", rotary=None,
                 interleaved=False, norm=True, scale=1.0, eps=1e-6, seed=0,
                 positions=None, values=True, pad=8, inv_freq=None):
        import torch
        t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        rng = np.random.default_rng(seed + N + heads + hd)
        self.kv, self.dtype = kv, dtype
        self.N, self.heads, self.kv_heads, self.hd = N, heads, kv_heads, hd
        self.rotary = hd if rotary is None else rotary
        self.interleaved, self.scale, self.eps = interleaved, scale, eps
        D = kv_heads * hd
        self.D, self.width = D, heads * hd
        self.rows = bits7(rng.standard_normal((N, self.width + 2 * D + pad)))
        self.norms = [bits7(1 + 0.3 * rng.standard_normal(hd)) if norm else
                      None for _ in range(2)]
        self.positions = (rng.integers(0, 40000, N) if positions is None
                          else np.asarray(positions))
        self.inv_freq = (np.asarray(kv.kvtc_rotary_frequencies(
            max(self.rotary, 2), 10000.0))[:self.rotary // 2]
            if inv_freq is None else np.asarray(inv_freq))
        self.num_blocks = max(1, -(-N // BLOCK)) + 2
        self.slots = rng.permutation(self.num_blocks * BLOCK)[:N]
        cuda = dict(device="cuda")
        self.d_rows = torch.from_numpy(self.rows).cuda().to(t)
        self.q = self.d_rows[:, :self.width]
        self.k = self.d_rows[:, self.width:self.width + D]
        self.v = self.d_rows[:, self.width + D:] if values else None
        self.d_norms = [None if w is None else torch.from_numpy(w).cuda()
                        .to(t) for w in self.norms]
        self.d_pos = torch.from_numpy(self.positions.astype(np.int32)).cuda()
        self.d_freq = torch.from_numpy(self.inv_freq.copy()).cuda()
        self.d_slots = torch.from_numpy(self.slots.astype(np.int64)).cuda()
        self.q_out = torch.full((N, self.width + 16), 77.0, dtype=t, **cuda)
        self.pools = [torch.full((self.num_blocks, BLOCK, D), 77.0, dtype=t,
                                 **cuda) for _ in range(2)]
        self.flags = torch.zeros(1, dtype=torch.int32, **cuda)

    def call(self, q_out=None, stream=None):
        out = self.q_out if q_out is None else q_out
        self.kv.kvtc_paged_rotate(
            self.N, self.heads, self.kv_heads, self.hd,
            {"bf16": 0, "fp16": 1}[self.dtype], self.q, self.k, self.v,
            self.d_rows.stride(0), self.d_pos if self.rotary else None,
            self.d_freq if self.rotary else None, self.rotary,
            self.interleaved, self.scale, self.d_norms[0], self.d_norms[1],
            self.eps, out, out.stride(0), self.d_slots, BLOCK,
            self.pools[0], self.pools[1] if self.v is not None else None,
            self.num_blocks, self.flags, stream=stream)

    def check(self, q_out=None, flags=0):
        N, hd = self.N, self.hd
        args = (self.positions, self.inv_freq, self.rotary, self.interleaved,
                self.scale, UNIT[self.dtype])
        w = self.width
        out = (self.q_out if q_out is None else q_out).double().cpu().numpy()
        y, tol = _chunks.rotate(self.rows[:, :w].reshape(N, -1, hd),
                                self.norms[0], self.eps, *args)
        near(out[:, :w].reshape(N, -1, hd), y, tol)
        if q_out is None:
            assert (out[:, w:] == 77).all()
        y, tol = _chunks.rotate(
            self.rows[:, w:w + self.D].reshape(N, -1, hd), self.norms[1],
            self.eps, *args)
        fine = (self.slots >= 0) & (self.slots < self.num_blocks * BLOCK)
        at = self.slots[fine]
        k, v = (p.double().cpu().numpy().reshape(-1, self.D)
                for p in self.pools)
        near(k[at].reshape(len(at), -1, hd), y[fine], tol[fine])
        if self.v is not None:
            np.testing.assert_array_equal(
                v[at], self.rows[fine, w + self.D:w + 2 * self.D])
        others = np.setdiff1d(np.arange(len(k)), at)
        assert (k[others] == 77).all() and (v[others] == 77).all()
        if self.v is None:
            assert (v == 77).all()
        assert int(self.flags.cpu()[0]) == flags


def near(x, y, tol):
    np.testing.assert_array_equal(np.isnan(x), np.isnan(y))
    fine = np.isfinite(y)
    far = np.abs(x - y)[fine] - tol[fine]
    assert far.size == 0 or far.max() <= 0, (
        f"{int((far > 0).sum())} of {far.size} further off than the bound, "
        f"worst by {far.max():.3g}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv_heads,hd", [
    (2, 2, 64), (5, 1, 64), (28, 4, 128), (7, 7, 128), (3, 1, 256),
    (32, 8, 128), (33, 3, 64)])
def test_head_layouts(kv, heads, kv_heads, hd, interleaved, dtype):
    a = Rotate(kv, 37, heads, kv_heads, hd, dtype, interleaved=interleaved)
    a.call()
    a.check()


@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 9, 100, 2431, 2433, 5000,
                               9800])
def test_numbers_of_tokens(kv, N):
    """Around one token a block and several (2432 at head_dim 256, 9728 at
    64)."""
    for hd in (64, 256):
        a = Rotate(kv, N, 2, 1, hd, norm=N % 2 == 0)
        a.call()
        a.check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,hd", [
    (0, 64), (8, 64), (24, 64), (56, 64), (0, 128), (32, 128), (72, 128),
    (120, 128), (8, 256), (64, 256), (248, 256)])
def test_part_of_the_head(kv, rotary, hd, interleaved):
    for norm in (False, True):
        a = Rotate(kv, 11, 6, 2, hd, rotary=rotary, interleaved=interleaved,
                   norm=norm, scale=1.25)
        a.call()
        a.check()


def test_far_and_negative_positions(kv):
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 131071, 999999937]
    a = Rotate(kv, len(at), 4, 2, 128, positions=at)
    a.call()
    a.check()
    # any angle per position, whole turns and negative ones among them
    f = np.linspace(-9, 9, 32)
    f[3] = 2 * np.pi
    a = Rotate(kv, 8, 2, 2, 64, positions=range(8), inv_freq=f, norm=False)
    a.call()
    a.check()


@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_in_place(kv, interleaved):
    a = Rotate(kv, 300, 12, 3, 128, interleaved=interleaved)
    a.call(q_out=a.d_rows)
    a.check(q_out=a.d_rows)
    # k and v beside them are as they were
    np.testing.assert_array_equal(
        a.d_rows[:, a.width:].double().cpu().numpy(), a.rows[:, a.width:])


def test_without_values_and_with_one_norm(kv):
    a = Rotate(kv, 20, 4, 2, 64, values=False)
    a.call()
    a.check()
    for i in range(2):
        a = Rotate(kv, 20, 4, 2, 128)
        a.norms[i] = a.d_norms[i] = None
        a.call()
        a.check()


def test_slots_outside(kv):
    a = Rotate(kv, 40, 4, 2, 64)
    a.slots[[3, 39]] = -1
    a.slots[5] = -2 ** 62
    a.d_slots.copy_(__import__("torch").from_numpy(a.slots))
    a.call()
    a.check()
    a.slots[7] = a.num_blocks * BLOCK
    a.slots[8] = 2 ** 62
    a.d_slots.copy_(__import__("torch").from_numpy(a.slots))
    for p in a.pools:
        p.fill_(77)
    a.call()
    a.check(flags=kv.KVTC_FLAG_BLOCK)


def test_zeros_infinities_and_nan(kv):
    a = Rotate(kv, 6, 4, 2, 64, rotary=32, eps=1e-6)
    hd = a.hd
    a.rows[0, :hd] = 0                      # a head of zeros: stays zero
    a.rows[1, hd + 3] = np.nan              # NaN fills its own head
    a.rows[2, a.width + 5] = np.nan
    a.d_rows.copy_(__import__("torch").from_numpy(a.rows))
    a.call()
    a.check()
    out = a.q_out.float().cpu().numpy()
    assert (out[0, :hd] == 0).all()
    assert np.isnan(out[1, hd:2 * hd]).all() and np.isfinite(
        out[1, 2 * hd:4 * hd]).all()


def test_graph_and_streams(kv):
    import torch
    a = Rotate(kv, 70, 8, 2, 128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.call()
    rng = np.random.default_rng(1)
    a.rows = bits7(rng.standard_normal(a.rows.shape))
    a.positions = rng.integers(0, 1000, a.N)
    a.slots = rng.permutation(a.num_blocks * BLOCK)[:a.N]
    a.d_rows.copy_(torch.from_numpy(a.rows))
    a.d_pos.copy_(torch.from_numpy(a.positions))
    a.d_slots.copy_(torch.from_numpy(a.slots))
    g.replay()
    a.check()
    b = Rotate(kv, 71, 8, 2, 128)
    st.wait_stream(torch.cuda.current_stream())
    b.call(stream=st)
    st.synchronize()
    b.check()


def test_pools_past_32_bits(kv):
    """Rows past 2^32 elements of a pool and of the tokens."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a = Rotate(kv, 5, 8, 8, 128, pad=0)
    blocks = (1 << 32) // (16 * a.D) + 8
    pool = torch.zeros((blocks, 16, a.D), dtype=torch.bfloat16,
                       device="cuda")
    a.slots = np.array([blocks * 16 - 1, blocks * 16 - 70, 0, 9, 11])
    a.d_slots.copy_(torch.from_numpy(a.slots))
    whole, a.num_blocks = a.pools, blocks
    a.pools = [pool, whole[1].new_zeros((blocks, 16, a.D))]
    a.call()
    y, tol = _chunks.rotate(
        a.rows[:, a.width:a.width + a.D].reshape(5, -1, a.hd), a.norms[1],
        a.eps, a.positions, a.inv_freq, a.rotary, False, 1.0, UNIT["bf16"])
    got = pool.view(-1, a.D)[a.d_slots].double().cpu().numpy()
    near(got.reshape(5, -1, a.hd), y, tol)
    got = a.pools[1].view(-1, a.D)[a.d_slots]
    assert torch.equal(got, a.v)
