"""A serving run with chunks: requests get blocks (kvtc_paged_assign), their
chunk's queries and keys are normed and rotated into the pools
(kvtc_paged_rotate) and attended (kvtc_paged_attend_chunks), the weight of each
cached token is gathered (kvtc_paged_weigh), long caches are cut in place
(kvtc_paged_evict), and decoding goes on over what is left
(kvtc_paged_attend); from captured graphs too (needs a GB300)."""
import numpy as np
import pytest

import _chunks
import _paged
from _chunks import check_chunks
from _paged import BLOCK, UNIT, bits7, blocks_of, check_attend, softmax_scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
def test_prompt_evict_decode(graph):
    import torch
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    H, KV, hd, keep, sink, window = 12, 3, 128, 96, 4, 16
    D, width, scale = KV * hd, H * hd, softmax_scale(hd)
    R, cols, cap = 4, 24, 256
    rng = np.random.default_rng(0)
    num_blocks = R * cols
    i32 = dict(dtype=torch.int32, device="cuda")
    i64 = dict(dtype=torch.int64, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    pool_k, pool_v = (torch.full((num_blocks, BLOCK, D), float("nan"), **bf)
                      for _ in "kv")
    free = torch.from_numpy(rng.permutation(num_blocks).astype(np.int32))
    free = free.cuda()
    head, held = torch.zeros(1, **i64), torch.zeros(R, **i32)
    lens, table = torch.zeros(R, **i32), torch.full((R, cols), -1, **i32)
    slots, cu = torch.empty(cap, **i64), torch.empty(R + 1, **i64)
    flags = torch.zeros(1, **i32)
    positions = torch.zeros(cap, **i32)
    freq = torch.tensor(kv.kvtc_rotary_frequencies(
        hd, 1e6, kv.KVTC_ROTARY_BANDS, 4.0, 8192.0, 1.0, 4.0),
        dtype=torch.float64, device="cuda")
    norms = [bits7(1 + 0.2 * rng.standard_normal(hd)) for _ in range(2)]
    d_norms = [torch.from_numpy(w).cuda().bfloat16() for w in norms]
    qkv = torch.zeros((cap, width + 2 * D), **bf)
    q, out = torch.zeros((cap, width), **bf), torch.zeros((cap, width), **bf)
    lse = torch.zeros((cap, H), device="cuda")
    acc = torch.zeros((R, cols * BLOCK), device="cuda")
    kept = torch.zeros((R, keep), **i32)
    ws = torch.empty(max(
        kv.kvtc_paged_assign_workspace_bytes(R),
        kv.kvtc_paged_attend_workspace_bytes(R, H, KV, hd),
        kv.kvtc_paged_attend_chunks_workspace_bytes(R, cap, H, KV, hd),
        kv.kvtc_paged_weigh_workspace_bytes(R, cap, H, KV, hd),
        kv.kvtc_paged_evict_workspace_bytes(R, cols)), dtype=torch.uint8,
        device="cuda")

    def step():
        kv.kvtc_paged_assign(R, held, lens, free, num_blocks, head, table,
                             cols, BLOCK, slots, cap, cu, held, head, ws,
                             ws.numel(), flags)
        kv.kvtc_paged_rotate(cap, H, KV, hd, 0, qkv, qkv[:, width:],
                             qkv[:, width + D:], qkv.stride(0), positions,
                             freq, hd, False, 1.0, d_norms[0], d_norms[1],
                             1e-6, q, width, slots, BLOCK, pool_k, pool_v,
                             num_blocks, flags)
        kv.kvtc_paged_attend_chunks(R, cap, H, KV, hd, 0, q, width, pool_k,
                                    pool_v, num_blocks, BLOCK, table, cols,
                                    cu, held, 0, 0, scale, out, width, lse,
                                    ws, ws.numel(), flags)
        kv.kvtc_paged_weigh(R, cap, H, KV, hd, 0, q, width, pool_k,
                            num_blocks, BLOCK, table, cols, cu, held, 0, 0,
                            scale, lse, 1.0, acc, acc, cols * BLOCK, ws,
                            ws.numel(), flags)

    def cut():
        kv.kvtc_paged_evict(R, acc, cols * BLOCK, held, keep, sink, window,
                            table, table, cols, BLOCK, [pool_k, pool_v], D,
                            num_blocks, kept, acc, held, ws, ws.numel(),
                            flags)

    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graphs = []
        for body in (step, cut):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                body()
            graphs.append(g.replay)
        step, cut = graphs

    seen = [0] * R                     # tokens of each request so far
    have = np.zeros(R, np.int64)       # of them in its cache
    weights = [np.zeros(0) for _ in range(R)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for news in ([120, 60, 1, 0], [80, 30, 40, 9], [1, 1, 1, 1],
                 [3, 0, 100, 1]):
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device="cuda"))
        rows = qkv.double().cpu().numpy()
        at = np.concatenate([np.arange(seen[r], seen[r] + n)
                             for r, n in enumerate(news)] or [[]])
        positions.zero_()
        positions[:len(at)] = torch.from_numpy(at)
        have = have + news
        lens.copy_(torch.from_numpy(have))
        step()
        torch.cuda.synchronize()
        assert held.tolist() == have.tolist()
        # the rows that the pools now hold, and the queries
        first = np.concatenate([[0], np.cumsum(news)])
        n = int(first[-1])
        args = (at, freq.cpu().numpy(), hd, False, 1.0, UNIT["bf16"])
        for x, w, got in ((rows[:n, :width], norms[0], q[:n]),
                          (rows[:n, width:width + D], norms[1],
                           pool_k.view(-1, D)[slots[:n]])):
            y, tol = _chunks.rotate(x.reshape(n, -1, hd), w, 1e-6, *args)
            far = np.abs(got.double().cpu().numpy().reshape(y.shape) - y)
            assert (far <= tol).all()
        assert torch.equal(pool_v.view(-1, D)[slots[:n]],
                           qkv[:n, width + D:])
        # attention and weights of the rows as they stand in the pools
        tab = table.cpu().numpy()
        ks, vs = (p.double().cpu().numpy() for p in (pool_k, pool_v))
        qs = q.double().cpu().numpy().reshape(cap, H, hd)
        ref = _chunks.attend_chunks(qs, ks, vs, tab, first, have, 0, 0, scale,
                                    UNIT["bf16"])
        check_chunks(out.double().cpu().numpy().reshape(cap, H, hd),
                     lse.double().cpu().numpy(), ref)
        before = np.zeros((R, cols * BLOCK))
        for r in range(R):
            before[r, :len(weights[r])] = weights[r]
        want, tol = _chunks.weigh(qs, ks, tab, first, have, 0, 0, scale,
                                  lse.cpu().numpy(), 1.0, before)
        got = acc.double().cpu().numpy()
        for r in range(R):
            h = have[r]
            assert (np.abs(got[r, :h] - want[r, :h]) <= tol[r, :h] +
                    1e-6 * want[r, :h]).all()
            assert (got[r, h:] == 0).all()
        # cut, in place
        table0, acc0 = tab.copy(), acc.cpu().numpy().copy()
        pools0 = [p.view(torch.int16).cpu().numpy().copy()
                  for p in (pool_k, pool_v)]
        cut()
        torch.cuda.synchronize()
        want = _chunks.evict(acc0, have, keep, sink, window, table0, table0,
                             pools0, True)
        np.testing.assert_array_equal(kept.cpu().numpy(), want[0])
        np.testing.assert_array_equal(held.cpu().numpy(), want[2])
        got = acc.cpu().numpy()
        for r in range(R):
            np.testing.assert_array_equal(got[r, :have[r]],
                                          want[1][r, :have[r]])
        for p, x in zip((pool_k, pool_v), want[3]):
            np.testing.assert_array_equal(p.view(torch.int16).cpu().numpy(),
                                          x)
        seen = [s + m for s, m in zip(seen, news)]
        have = want[2].astype(np.int64)
        weights = [got[r, :have[r]].astype(np.float64) for r in range(R)]
    # one token a request over what is left
    qs = q[:R].contiguous()
    kv.kvtc_paged_attend(R, H, KV, hd, 0, qs, width, pool_k, pool_v,
                         num_blocks, BLOCK, table, cols, held, 0, 0, scale,
                         out, width, lse, ws, ws.numel(), flags)
    ref = _paged.attend(qs.double().cpu().numpy().reshape(R, H, hd),
                        pool_k.double().cpu().numpy(),
                        pool_v.double().cpu().numpy(), table.cpu().numpy(),
                        have, 0, 0, scale, UNIT["bf16"])
    check_attend(out[:R].double().cpu().numpy().reshape(R, H, hd),
                 lse[:R].double().cpu().numpy(), ref)
    assert int(flags.cpu()[0]) == 0
    assert int(head.cpu()[0]) <= num_blocks and blocks_of(keep) == 6
