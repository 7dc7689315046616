"""One serving step over a restored cache: requests get their blocks
(kvtc_paged_assign), their compressed prefixes are restored into them
(kvtc_decompress_paged), new tokens' rows are appended through the slots
(kvtc_paged_append) and attended (kvtc_paged_attend), layer by layer, from
captured graphs too (needs a GB300)."""
import numpy as np
import pytest

import _paged
import synth
from _paged import BLOCK, blocks_of, check_attend, softmax_scale
from _parity import blob_for, calibrate_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
def test_restore_append_and_attend(graph):
    import torch
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    name = "qwen25_7b_paged"
    w = synth.WORKLOADS[name]
    layers, steps = 2, 20
    pairs = [(l, k) for l in range(layers) for k in range(2)]
    calib = kv.kvtc_calib_load(blob_for(name, calibrate_workload(name,
                                                                 pairs)), 0)
    D, hd, heads = w.D, w.head_dim, 28
    prefix = [700, 150, 47, 1]
    R = len(prefix)
    # compressed prefixes, and the dense rows that the restore gives
    streams, dense = [], [[None] * R for _ in pairs]
    for r, T in enumerate(prefix):
        x = [synth.eval_tokens_torch(w, l, k, r, T) for l, k in pairs]
        n = sum(calib.stream_bytes(l, k, T) for l, k in pairs)
        comp = torch.empty(n, dtype=torch.uint8, device="cuda")
        kv.kvtc_compress(calib, 0, layers, 3, x, D, T, comp, n)
        back = [torch.empty_like(y) for y in x]
        kv.kvtc_decompress(calib, 0, layers, 3, comp, n, T, back, D)
        streams.append(comp)
        for i, y in enumerate(back):
            dense[i][r] = y
    cols = blocks_of(max(prefix) + steps)
    num_blocks = sum(blocks_of(T + steps) for T in prefix) + 2
    free = torch.from_numpy(np.random.default_rng(1).permutation(num_blocks)
                            .astype(np.int32)).cuda()
    pools = [torch.full((num_blocks, BLOCK, D), float("nan"),
                        dtype=torch.bfloat16, device="cuda") for _ in pairs]
    table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    lens = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    head = torch.zeros(1, dtype=torch.int64, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.empty(R + 1, dtype=torch.int64, device="cuda")
    many = torch.empty(sum(prefix), dtype=torch.int64, device="cuda")
    slots = torch.empty(R, dtype=torch.int64, device="cuda")
    ws = torch.empty(max(kv.kvtc_paged_assign_workspace_bytes(R),
                         kv.kvtc_paged_attend_workspace_bytes(
                             R, heads, w.heads, hd)),
                     dtype=torch.uint8, device="cuda")

    def assign(to):
        kv.kvtc_paged_assign(R, held, lens, free, num_blocks, head, table,
                             cols, BLOCK, to, to.numel(), cu, held, head, ws,
                             ws.numel(), flags)

    assign(many)
    kv.kvtc_decompress_paged(calib, 0, layers, 3, streams, prefix, table,
                             cols, BLOCK, pools, num_blocks)
    # the slots name the rows that the restore wrote
    for i in range(len(pairs)):
        got = pools[i].view(-1, D)[many]
        assert torch.equal(got, torch.cat(dense[i]))

    qkv = [torch.empty((R, heads * hd + 2 * D), dtype=torch.bfloat16,
                       device="cuda") for _ in range(layers)]
    outs = [torch.empty((R, heads * hd), dtype=torch.bfloat16, device="cuda")
            for _ in range(layers)]
    lses = [torch.empty((R, heads), device="cuda") for _ in range(layers)]
    wide = qkv[0].shape[1]

    def step():
        torch.add(held, 1, out=lens)
        assign(slots)
        for l in range(layers):
            k, v = (qkv[l][:, heads * hd + i * D:heads * hd + (i + 1) * D]
                    for i in range(2))
            kv.kvtc_paged_append([k, v], wide, R, slots, D, BLOCK,
                                 pools[2 * l:2 * l + 2], num_blocks, flags)
            kv.kvtc_paged_attend(R, heads, w.heads, hd, kv.KVTC_DTYPE_BF16,
                                 qkv[l], wide, pools[2 * l],
                                 pools[2 * l + 1], num_blocks, BLOCK, table,
                                 cols, held, 0, 0, softmax_scale(hd),
                                 outs[l], heads * hd, lses[l], ws,
                                 ws.numel(), flags)

    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
        one = g.replay
    else:
        one = step
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for s in range(steps):
        for l in range(layers):
            qkv[l].copy_(torch.randn(qkv[l].shape, generator=gen,
                                     device="cuda"))
        one()
        torch.cuda.synchronize()
        for l in range(layers):
            for i in range(2):
                rows = qkv[l][:, heads * hd + i * D:heads * hd + (i + 1) * D]
                for r in range(R):
                    dense[2 * l + i][r] = torch.cat(
                        [dense[2 * l + i][r], rows[r:r + 1]])
            if s not in (0, steps - 1):
                continue
            for r in range(R):
                n = prefix[r] + s + 1
                pad = blocks_of(n) * BLOCK
                k, v = (torch.nn.functional.pad(
                    dense[2 * l + i][r].double(), (0, 0, 0, pad - n)).view(
                        -1, BLOCK, D).cpu().numpy() for i in range(2))
                q = qkv[l][r:r + 1, :heads * hd].double().cpu().numpy()
                ref = _paged.attend(q.reshape(1, heads, hd), k, v,
                                    np.arange(pad // BLOCK)[None], [n], 0, 0,
                                    softmax_scale(hd), _paged.UNIT["bf16"])
                check_attend(
                    outs[l][r].double().cpu().numpy().reshape(1, heads, hd),
                    lses[l][r].double().cpu().numpy()[None], ref)
    assert int(flags.cpu()[0]) == 0
    assert int(head.cpu()[0]) == sum(blocks_of(T + steps) for T in prefix)
    calib.free()


FIRST_CALLS = """
import numpy as np, torch
import kv_cache_transform_gb300 as kv
R, H, KV, hd, cols, nb = 3, 8, 2, 128, 4, 16
D = KV * hd
i32 = dict(dtype=torch.int32, device='cuda')
i64 = dict(dtype=torch.int64, device='cuda')
pools = [torch.zeros(nb, 16, D, dtype=torch.bfloat16, device='cuda')
         for _ in range(2)]
table, held = torch.full((R, cols), -1, **i32), torch.zeros(R, **i32)
lens = torch.tensor([20, 1, 33], **i32)
free, head = torch.arange(nb, **i32), torch.zeros(1, **i64)
cap = {cap}
slots, cu = torch.empty(cap, **i64), torch.empty(R + 1, **i64)
flags = torch.zeros(1, **i32)
ws = torch.empty(max(kv.kvtc_paged_assign_workspace_bytes(R),
                     kv.kvtc_paged_attend_workspace_bytes(R, H, KV, hd)),
                 dtype=torch.uint8, device='cuda')
rows = torch.randn(cap, 2 * D, device='cuda').bfloat16()
q = torch.randn(R, H * hd, device='cuda').bfloat16()
out, lse = torch.empty_like(q), torch.empty(R, H, device='cuda')
st = torch.cuda.Stream()
st.wait_stream(torch.cuda.current_stream())
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=st):
    kv.kvtc_paged_assign(R, held, lens, free, nb, head, table, cols, 16,
                         slots, cap, cu, held, head, ws, ws.numel(), flags)
    kv.kvtc_paged_append([rows[:, :D], rows[:, D:]], 2 * D, cap, slots, D, 16,
                         pools, nb, flags)
    kv.kvtc_paged_attend(R, H, KV, hd, kv.KVTC_DTYPE_BF16, q, H * hd,
                         pools[0], pools[1], nb, 16, table, {cols}, held, 0,
                         0, hd ** -0.5, out, H * hd, lse, ws, ws.numel(),
                         flags)
g.replay()
torch.cuda.synchronize()
assert int(flags[0]) == 0 and held.tolist() == [20, 1, 33]
at = 0
for r, n in enumerate((20, 1, 33)):
    k = rows[at:at + n, :D].double().view(n, KV, hd)
    v = rows[at:at + n, D:].double().view(n, KV, hd)
    x = q[r].double().view(KV, 4, hd) @ k.permute(1, 2, 0) * hd ** -0.5
    ref = (torch.softmax(x, -1) @ v.permute(1, 0, 2)).reshape(-1)
    assert (out[r].double() - ref).abs().max() <= 2 ** -8 * ref.abs().max()
    at += n
print('captured first')
"""


@pytest.mark.parametrize("cap", [54, 5000])
def test_first_calls_of_a_process_are_captured(cap):
    """Nothing has to run before a capture: a process whose first calls are
    inside one (both launch forms of assign)."""
    import os
    import subprocess
    import sys
    from kv_cache_transform_gb300 import _build
    _build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run(
        [sys.executable, "-c", FIRST_CALLS.format(cap=cap, cols="cols")],
        cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, \
        r.stdout[-2000:] + r.stderr[-4000:]
