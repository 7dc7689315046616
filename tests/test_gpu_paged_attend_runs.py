"""kvtc_paged_attend where its pages are dealt out to all blocks in equal runs
and parts are joined by a second launch, on the GPU against the plain form in
64 bits (needs a GB300).

Few items (request, KV head, tile of query heads) under a narrow table take
the clusters instead; each test here says which form it means, and the number
of launches shows that it was that one."""
import numpy as np
import pytest

import _paged
from _paged import BLOCK, blocks_of, paged_case
from test_gpu_paged_attend import Attend

pytestmark = pytest.mark.gpu

RUNS, CLUSTERS = 2, 1           # launches of a call


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


class Formed(Attend):
    """A call that must take the given form."""

    def __init__(self, kv, case, form=RUNS, **more):
        super().__init__(kv, *case, **more)
        self.form = form

    def call(self, **more):
        n = self.kv.kvtc_launch_count()
        super().call(**more)
        assert self.kv.kvtc_launch_count() - n == self.form

    def bits(self):
        """Everything that the call writes, zeros' signs among it."""
        import torch
        return (self.out.view(torch.int16).clone(),
                self.lse.view(torch.int32).clone())


def ragged(rng, R, longest=700):
    """Lengths whose items lie in one warp's run, over two warps', over a
    block and over several."""
    lens = rng.integers(0, 120, R)
    lens[rng.integers(0, R, R // 8)] = 0
    lens[rng.integers(0, R, 3)] = rng.integers(longest // 2, longest, 3)
    lens[R // 2] = longest
    lens[[1, R - 1]] = 1, 33
    return lens


def case(seed, lens, heads, kv_heads, hd, columns=0):
    q, k, v, table, lens = paged_case(seed, lens, heads, kv_heads, hd)
    if columns > table.shape[1]:
        table = np.pad(table, ((0, 0), (0, columns - table.shape[1])),
                       constant_values=2 ** 31 - 1)
    return q, k, v, table, lens


# (query heads, KV heads, head_dim): one, two and four tiles of eight heads a
# warp, groups of one and of several such tiles
LAYOUTS = [(8, 4, 64), (48, 4, 64), (80, 4, 64), (160, 4, 64),
           (28, 4, 128), (48, 4, 128), (80, 4, 128),
           (8, 4, 256), (48, 4, 256), (72, 4, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,hd", LAYOUTS)
def test_head_layouts(kv, heads, kv_heads, hd, dtype):
    rng = np.random.default_rng(heads + hd)
    a = Formed(kv, case(heads + hd, ragged(rng, 43), heads, kv_heads, hd),
               dtype=dtype)
    a.call()
    a.check()


@pytest.mark.parametrize("heads,kv_heads,hd,R,longest", [
    (4, 2, 64, 3, 9001), (24, 2, 64, 3, 9001), (40, 2, 64, 3, 5000),
    (8, 2, 128, 2, 9001), (24, 2, 128, 3, 5000), (8, 2, 256, 3, 5000),
    (24, 2, 256, 2, 3001), (8, 1, 64, 1, 70001), (16, 1, 256, 1, 5000),
    (8, 1, 128, 19, 900), (16, 1, 128, 19, 900), (8, 1, 256, 19, 600)])
def test_few_long_items_under_a_wide_table(kv, heads, kv_heads, hd, R,
                                           longest):
    """Items over up to all blocks: the join across blocks by groups of
    warps."""
    rng = np.random.default_rng(longest + hd)
    lens = rng.integers(0, longest, R)
    lens[R // 2] = longest
    a = Formed(kv, case(R + longest, lens, heads, kv_heads, hd, 30000))
    a.call()
    a.check()


@pytest.mark.parametrize("heads,kv_heads,hd", [
    (8, 4, 64), (80, 4, 64), (28, 4, 128), (48, 4, 128), (8, 4, 256),
    (48, 4, 256)])
@pytest.mark.parametrize("sink,window", [
    (0, 1), (0, 23), (3, 40), (8, 16), (9, 100), (17, 7), (40, 61)])
def test_sink_and_window(kv, sink, window, heads, kv_heads, hd):
    """Windows that begin at every token of a page; what is not attended is
    infinite or NaN and its blocks have no place."""
    rng = np.random.default_rng(sink + window + hd)
    R = 48
    lens = sink + window + 40 + np.arange(R)     # each residue three times
    lens[-9:] = [0, 1, 5, sink, sink + 1, window, sink + window,
                 sink + window + 1, 611]
    q, k, v, table, lens = paged_case(sink + window, rng.permutation(lens),
                                      heads, kv_heads, hd)
    for r, n in enumerate(lens):
        seen = _paged.attended(n, sink, window)
        t = np.setdiff1d(np.arange(n), seen)
        k[table[r, t // BLOCK], t % BLOCK] = np.inf
        v[table[r, t // BLOCK], t % BLOCK] = np.nan
        gone = np.setdiff1d(np.arange(blocks_of(n)), seen // BLOCK)
        table[r, gone] = -5
    a = Formed(kv, (q, k, v, table, lens), sink=sink, window=window)
    a.call()
    a.check()


@pytest.mark.parametrize("columns,form", [(0, RUNS), (30000, RUNS),
                                          (0, CLUSTERS)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_infinities_and_nan_in_attended_tokens(kv, hd, columns, form):
    """In one part of an item of several, in all of them, in short ones."""
    few = columns or form == CLUSTERS
    lens = [700, 700, 700, 700, 3, 700, 90, 700]
    lens = lens if few else lens + list(range(20, 100, 2))
    q, k, v, table, lens = case(hd, lens, 8, 4, hd, columns)
    q[:, :, 0] = 1.0

    def row(pool, r, t, head):
        return pool[table[r, t // BLOCK], t % BLOCK,
                    head * hd:(head + 1) * hd]
    row(k, 0, 20, 0)[0] = -np.inf           # a weight of zero
    row(k, 1, 350, 1)[5] = np.nan           # NaN for KV head 1 alone
    row(v, 2, 699, 0)[7] = np.inf           # an infinite channel
    row(v, 3, 0, 1)[9] = np.nan             # a NaN channel
    for t in range(3):
        row(k, 4, t, 1)[0] = -np.inf        # every weight is zero
    row(k, 5, 400, 0)[0] = np.inf           # s = +inf: inf - inf
    for t in range(90):
        row(k, 6, t, 2)[0] = -np.inf
    for t in range(640):                    # the whole of some parts
        row(k, 7, t, 3)[0] = -np.inf
    with np.errstate(all="ignore"):
        a = Formed(kv, (q, k, v, table, lens), form)
        a.call()
        out, lse, tol, tl = a.reference()
    assert np.isnan(out[1, 2:4]).all() and np.isfinite(out[1, :2]).all()
    assert (lse[4, 2:4] == -np.inf).all() and (out[4, 2:4] == 0).all()
    assert (lse[6, 4:6] == -np.inf).all() and np.isfinite(lse[7]).all()
    # where the maximum is +inf the formula gives NaN throughout
    out[5, :2] = lse[5, :2] = np.nan
    a.check((out, lse, tol, tl))


@pytest.mark.parametrize("columns", [0, 30000])
def test_bad_block_ids_are_left_out_and_flagged(kv, columns):
    few = columns > 0
    lens = [900, 40, 64, 16, 500] + ([] if few else list(range(1, 160, 4)))
    q, k, v, clean, lens = case(24, lens, 12, 4, 128, columns)
    for cut in (slice(0, 1), slice(1, 30), slice(20, 21), slice(0, 56),
                slice(0, 57)):
        table = clean.copy()
        table[0, cut] = -1
        table[1, 1], table[2, 3] = k.shape[0], 2 ** 31 - 1
        table[3, 0] = -2 ** 31               # nothing is left of it
        table[4, 3:25:2] = -9
        a = Formed(kv, (q, k, v, table, lens))
        a.call()
        a.check(flags=kv.KVTC_FLAG_BLOCK)
        assert (a.out[3, :a.width] == 0).all()
    b = Formed(kv, (q, k, v, clean, lens))
    b.call()
    b.check()


def test_lengths_outside_the_table(kv):
    lens = [48] * 50 + [30, 7]
    q, k, v, table, lens = paged_case(25, lens, 8, 4, 64, extra_cols=0)
    table[50, 2] = table[51, 1] = table[51, 2] = 0
    ask = lens.copy()
    ask[[3, 20]] = 1000, 2 ** 31 - 1
    ask[50] = -9
    a = Formed(kv, (q, k, v, table, ask))
    a.call()
    a.check(flags=kv.KVTC_FLAG_SPACE)


@pytest.mark.parametrize("form", [RUNS, CLUSTERS])
@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127])
def test_the_largest_scale(kv, scale, form):
    """Scores of zero stay zero beside a scale near fp32's largest, and
    products of 2^-122 with it are of order 32."""
    q, k, v, table, lens = case(50, [90] * (60 if form == RUNS else 2), 8, 4,
                                64)
    k[:, :, 64:] *= 2.0 ** -60
    q[:, 2:] *= 2.0 ** -62               # KV heads 1 to 3
    q[:, :2] = 0.0                       # KV head 0: every score is zero
    a = Formed(kv, (q, k, v, table, lens), form, scale=scale)
    a.call()
    a.check()


def many(seed, R=64, longest=2000, columns=0, heads=28, kv_heads=4, hd=128):
    rng = np.random.default_rng(seed)
    return case(seed, ragged(rng, R, longest), heads, kv_heads, hd, columns)


@pytest.mark.parametrize("what", [
    "many", "windows", "few long", "short", "two heads' tiles", "fp16",
    "clusters"])
def test_repeated_calls_give_equal_bits(kv, what):
    """Which warp joins two parts is a matter of timing, and what the
    workspace holds is of no matter."""
    import torch
    more, form = {}, RUNS
    if what == "few long":
        c = case(30, [9000, 3, 812, 0, 640], 28, 4, 128, 30000)
    elif what == "short":
        c = many(31, R=500, longest=60)
    elif what == "two heads' tiles":
        c = many(32, R=40, heads=48, hd=256)
    elif what == "clusters":
        c, form = case(33, [5000, 3, 812, 0, 64], 28, 4, 128), CLUSTERS
    else:
        c = many(34, R=100)
        more = {"windows": dict(sink=4, window=50),
                "fp16": dict(dtype="fp16")}.get(what, {})
    a = Formed(kv, c, form, **more)
    a.call()
    a.check()
    first = a.bits()
    burn = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(40):
        a.out.fill_(77.0)
        a.lse.fill_(77.0)
        a.ws.random_(0, 256)
        if i % 2:
            burn.random_(0, 256)            # pages from HBM, not from L2
        a.call()
        for x, y in zip(a.bits(), first):
            assert torch.equal(x, y)


def test_equal_bits_where_an_output_is_zero(kv):
    """Sums of negative and of zero terms, whose earlier parts vanish beside
    the last: zeros have one sign, whoever joins the parts."""
    import torch
    R, hd, n = 1700, 64, 48
    q = np.zeros((R, 1, hd))
    q[:, :, 0] = 1.0
    k = np.zeros((3 * R, BLOCK, hd))
    v = np.full((3 * R, BLOCK, hd), -1.0)
    table = np.arange(3 * R, dtype=np.int32).reshape(R, 3)
    k[2::3, :, 0] = 400.0
    v[2::3] = -0.0
    lens = np.full(R, n, np.int32)
    a = Formed(kv, (q, k, v, table, lens), scale=1.0)
    a.call()
    a.check()
    first = a.bits()
    for i in range(30):
        a.out.fill_(77.0)
        a.ws.random_(0, 256)
        a.call()
        for x, y in zip(a.bits(), first):
            assert torch.equal(x, y), int((x != y).sum())


def capture(call):
    import torch
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    return g


@pytest.mark.parametrize("R,columns", [(64, 0), (4, 30000), (300, 0)])
def test_replayed_from_a_graph_with_other_inputs(kv, R, columns):
    import torch
    q, k, v, table, lens = many(41, R, 900, columns)
    a = Formed(kv, (q, k, v, table, lens))
    g = capture(a.call)
    rng = np.random.default_rng(0)
    for i in range(4):
        lens2 = np.minimum(lens, rng.integers(0, 900, R)).astype(np.int32)
        order = rng.permutation(R)
        q2 = _paged.bits7(rng.standard_normal(q.shape))
        a.set_q(q2)
        a.lens.copy_(torch.from_numpy(lens2[order]).cuda())
        a.table.copy_(torch.from_numpy(table[order]).cuda())
        a.ws.random_(0, 256)
        g.replay()
        torch.cuda.synchronize()
        a.check(a.reference(q=q2, lens=lens2[order], table=table[order]))


def test_graphs_that_share_a_workspace(kv):
    """Captured apart, replayed in turn on one stream: two of this form, of
    other shapes, and one of clusters."""
    import torch
    calls = [Formed(kv, many(42)),
             Formed(kv, case(43, [4000, 1900], 16, 2, 64, 30000),
                    dtype="fp16"),
             Formed(kv, case(44, [700, 2, 90], 8, 2, 128), CLUSTERS),
             Formed(kv, many(45, 40, 500, heads=48, hd=256))]
    ws = max((c.ws for c in calls), key=lambda w: w.numel())
    graphs = [capture(lambda c=c: c.call(ws=ws)) for c in calls]
    for c in calls:
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
    for i in (0, 1, 1, 3, 0, 2, 1, 0, 3):
        graphs[i].replay()
    torch.cuda.synchronize()
    for c in calls:
        c.check()


def test_calls_at_once_on_two_streams(kv):
    import torch
    calls = [Formed(kv, many(46)),
             Formed(kv, case(47, [40, 6000], 8, 2, 128, 30000)),
             Formed(kv, many(48, 80, 300, hd=64))]
    streams = [torch.cuda.Stream() for _ in calls]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, st in zip(calls, streams):
            c.call(stream=st)
    torch.cuda.synchronize()
    for c in calls:
        c.check()


@pytest.mark.parametrize("form", [RUNS, CLUSTERS])
def test_captured_behind_a_long_copy_on_another_stream(kv, form):
    """The copy of a K pool of 300 MB on a second stream ends last, just
    before the call: a kernel that began to read too early would read NaN.
    The requests' pages are the pool's last."""
    import torch
    rng = np.random.default_rng(5)
    lens = ragged(rng, 64, 900) if form == RUNS else [300, 20, 90, 1]
    q, k, v, table, lens = case(49, lens, 28 if form == RUNS else 8,
                                4 if form == RUNS else 2, 128)
    a = Formed(kv, (q, k, v, table, lens), form)
    nb, (_, _, width) = k.shape[0], k.shape
    blocks = (300 << 20) // (BLOCK * width * 2)
    assert blocks > nb
    small_k, small_v = a.k, a.v
    a.k = torch.full((blocks, BLOCK, width), float("nan"),
                     dtype=small_k.dtype, device="cuda")
    a.v, k_in = torch.zeros_like(a.k), torch.zeros_like(a.k)
    a.v[-nb:], k_in[-nb:] = small_v, small_k
    a.table.copy_(torch.where(a.table < nb, a.table + (blocks - nb),
                              a.table))
    a.num_blocks = blocks
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    lens_in = a.lens.clone()
    with torch.cuda.graph(g, stream=main):
        a.out.fill_(77.0)
        a.lens.copy_(lens_in)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a.k.copy_(k_in)
        main.wait_stream(side)
        a.call()
        a.k[-nb:].fill_(float("nan"))
        a.lens.zero_()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        a.check()
        assert (a.lens == 0).all()


@pytest.mark.parametrize("columns", [0, 30000])
def test_serving_steps(kv, columns):
    """Requests are admitted, their prompts appended and attended, and steps
    of one token replayed from a graph, the state in place: many requests,
    and few under a wide table."""
    import torch
    heads, kv_heads, hd, steps = 28, 4, 128, 18
    rng = np.random.default_rng(6)
    prompt = rng.integers(1, 200, 44) if not columns else \
        np.array([700, 33, 1])
    R, D = len(prompt), kv_heads * hd
    cols = max(columns, blocks_of(int(prompt.max()) + steps))
    total = int(prompt.sum()) + steps * R
    nb = int(sum(blocks_of(int(n) + steps) for n in prompt)) + 2
    i32, i64 = (dict(dtype=t, device="cuda") for t in (torch.int32,
                                                       torch.int64))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rows = torch.randn((total, (heads + 2 * kv_heads) * hd), generator=gen,
                       device="cuda").bfloat16()
    k_rows, v_rows = (rows[:, heads * hd + i * D:heads * hd + (i + 1) * D]
                      for i in range(2))
    wide = rows.shape[1]
    pools = [torch.full((nb, BLOCK, D), float("nan"), dtype=torch.bfloat16,
                        device="cuda") for _ in range(2)]
    free = torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    table, held = torch.full((R, cols), -1, **i32), torch.zeros(R, **i32)
    lens = torch.from_numpy(prompt.astype(np.int32)).cuda()
    head, flags = torch.zeros(1, **i64), torch.zeros(1, **i32)
    cu = torch.empty(R + 1, **i64)
    first = torch.empty(int(prompt.sum()), **i64)
    slots = torch.empty(R, **i64)
    ws = torch.empty(max(kv.kvtc_paged_assign_workspace_bytes(R),
                         kv.kvtc_paged_attend_workspace_bytes(
                             R, heads, kv_heads, hd)),
                     dtype=torch.uint8, device="cuda")
    step_rows = torch.empty((R, wide), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((R, heads * hd), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, heads), device="cuda")

    def assign(to):
        kv.kvtc_paged_assign(R, held, lens, free, nb, head, table, cols,
                             BLOCK, to, to.numel(), cu, held, head, ws,
                             ws.numel(), flags)

    assign(first)
    n0 = first.numel()
    kv.kvtc_paged_append([k_rows, v_rows], wide, n0, first, D, BLOCK, pools,
                         nb, flags)

    def step():
        torch.add(held, 1, out=lens)
        assign(slots)
        kv.kvtc_paged_append(
            [step_rows[:, heads * hd:heads * hd + D],
             step_rows[:, heads * hd + D:]], wide, R, slots, D, BLOCK, pools,
            nb, flags)
        n = kv.kvtc_launch_count()
        kv.kvtc_paged_attend(R, heads, kv_heads, hd, kv.KVTC_DTYPE_BF16,
                             step_rows, wide, pools[0], pools[1], nb, BLOCK,
                             table, cols, held, 0, 0, hd ** -0.5, out,
                             heads * hd, lse, ws, ws.numel(), flags)
        assert kv.kvtc_launch_count() - n == RUNS

    g = capture(step)
    at = np.concatenate([[0], np.cumsum(prompt)])
    own = [[*range(at[r], at[r + 1])] for r in range(R)]
    for s in range(steps):
        a = n0 + s * R
        step_rows.copy_(rows[a:a + R])
        g.replay()
        for r in range(R):
            own[r].append(a + r)
        if s not in (0, 7, steps - 1):
            continue
        torch.cuda.synchronize()
        # the rows of all requests, in pages of their own
        lens_now = [len(x) for x in own]
        pages = np.full((R, cols), 2 ** 31 - 1, np.int64)
        many_k, many_v, b = [], [], 0
        for r, idx in enumerate(own):
            n, pad = len(idx), blocks_of(len(idx)) * BLOCK
            for src, to in ((k_rows, many_k), (v_rows, many_v)):
                x = np.full((pad, D), np.nan)
                x[:n] = src[idx].double().cpu().numpy()
                to.append(x.reshape(-1, BLOCK, D))
            pages[r, :pad // BLOCK] = np.arange(b, b + pad // BLOCK)
            b += pad // BLOCK
        q = step_rows[:, :heads * hd].double().cpu().numpy()
        ref = _paged.attend(q.reshape(R, heads, hd), np.concatenate(many_k),
                            np.concatenate(many_v), pages, lens_now, 0, 0,
                            hd ** -0.5, _paged.UNIT["bf16"])
        _paged.check_attend(
            out.double().cpu().numpy().reshape(R, heads, hd),
            lse.double().cpu().numpy(), ref)
    assert int(flags.cpu()[0]) == 0
    assert held.tolist() == [len(x) for x in own]
