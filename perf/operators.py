"""Cases of the paged-cache operators: blocks and slots for requests, rows of
new tokens written through the slots, attention of one new token per request.

``own`` false: the operators in plain torch operations.  ``own`` true: the
calls a user makes of ``kv_cache_transform_gb300``.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16           # tokens per block of the paged pools
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _assign(name, requests, lo, hi, step):
    """step: new tokens of each request; 0: every request is new."""
    return {"name": name, "op": "assign", "requests": requests, "lo": lo,
            "hi": hi, "step": step}


def _append(name, tokens, width, streams):
    return {"name": name, "op": "append", "tokens": tokens, "width": width,
            "streams": streams}


def _attend(name, requests, lo, hi, heads, kv_heads, head_dim, dtype="bf16",
            sink=0, window=0):
    return {"name": name, "op": "attend", "requests": requests, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "sink": sink,
            "window": window}


def listed():
    return [
        # one decode step of the 64-request paged workload: one slot each,
        # a block for every request whose last block is full
        _assign("assign_decode_64", 64, 1, 4096, 1),
        # admission of that workload's 64 requests, ragged
        _assign("assign_prefill_64x4k", 64, 1, 4096, 0),
        # admission of a large batch at the longest context (32768)
        _assign("assign_prefill_128x32k", 128, 1000, 32768, 0),
        # the K and V rows of one decode step of 64 requests (D = 512)
        _append("append_decode_64", 64, 512, 2),
        # the K and V rows of an 8192-token prompt, one layer (D = 1024)
        _append("append_prefill_8k", 8192, 1024, 2),
        # the smallest shape: two heads of 64, 256 tokens; latency alone
        _attend("attend_tiny_256", 1, 256, 256, 2, 2, 64),
        # one request at 8K and at 32K, four query heads a KV head
        _attend("attend_1x8k_g4", 1, 8192, 8192, 32, 8, 128),
        _attend("attend_1x32k_g4", 1, 32768, 32768, 32, 8, 128),
        # the 64-request paged workload, ragged, seven query heads a KV head
        _attend("attend_64x4k_g7", 64, 1, 4096, 28, 4, 128),
        # a batch of long requests, eight query heads a KV head
        _attend("attend_16x16k_g8", 16, 1000, 16384, 64, 8, 128),
        # sink and window tokens only (the codec's 4 and 128), many requests
        _attend("attend_window_256", 256, 1, 4096, 32, 8, 128, sink=4,
                window=128),
        # a head of its own for every query head (D = 8192), fp16
        _attend("attend_8x600_mha", 8, 37, 600, 64, 64, 128, "fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "attend", "attend"])
    if op == "assign":
        hi = _log_int(rng, 1, 32768)
        most = max(1, min(4096, 4000000 // hi))
        return _drop_name(_assign("", _log_int(rng, 1, most),
                                  rng.randint(1, hi), hi,
                                  rng.choice([0, 0, 1, rng.randint(1, 64)])))
    if op == "append":
        width = 64 * _log_int(rng, 1, 64)
        most = max(1, min(16384, (1 << 24) // width))
        return _drop_name(_append("", _log_int(rng, 1, most), width,
                                  rng.choice([1, 2, 2, 8])))
    head_dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
    width = head_dim * kv_heads
    hi = _log_int(rng, 1, 32768)
    most = max(1, min(1024, (1 << 28) // (hi * width)))
    sink, window = rng.choice([(0, 0), (0, 0), (0, 0),
                               (rng.randint(0, 40), _log_int(rng, 1, 4096))])
    return _drop_name(_attend("", _log_int(rng, 1, most), rng.randint(0, hi),
                              hi, kv_heads * group, kv_heads, head_dim,
                              rng.choice(["bf16", "bf16", "fp16"]), sink,
                              window))


def _drop_name(case):
    del case["name"]
    return case


def _lengths(case):
    """The requests' lengths in no order: spread evenly from lo to hi, so
    that their sum is the case's and not the seed's."""
    n, lo, hi = case["requests"], case["lo"], case["hi"]
    if n == 1:
        return np.array([hi], np.int64)
    return lo + (hi - lo) * np.arange(n, dtype=np.int64) // (n - 1)


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def _attended(case, lens):
    if not case["window"]:
        return lens
    return np.minimum(lens, case["sink"] +
                      np.minimum(lens, case["window"]))


def work(case):
    if case["op"] == "append":
        rows = case["tokens"] * case["width"] * case["streams"] * 2
        return {"bytes": 2 * rows + 8 * case["tokens"], "flops": 0}
    lens = _lengths(case)
    n = case["requests"]
    if case["op"] == "assign":
        held = np.maximum(lens - case["step"], 0) if case["step"] else 0 * lens
        tokens = int((lens - held).sum())
        blocks = int((_blocks(lens) - _blocks(held)).sum())
        # lengths in and out, offsets; a block id in and out; a slot
        return {"bytes": 20 * n + 8 * blocks + 8 * tokens, "flops": 0}
    tokens = int(_attended(case, lens).sum())
    width = case["kv_heads"] * case["head_dim"]
    rows = n * case["heads"] * case["head_dim"]
    blocks = int(_blocks(_attended(case, lens)).sum())
    return {"bytes": 4 * tokens * width + 4 * rows + 4 * n * case["heads"] +
            4 * blocks + 4 * n,
            "flops": 4 * case["heads"] * case["head_dim"] * tokens}


# ---------------------------------------------------------------- prepare
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, width, dtype, outliers):
    """Rows with a mean, a decaying low-rank part, a little noise and, for
    keys, four channels ten times as large: the shape of cached K and V."""
    mean = torch.randn(width, generator=g, device="cuda")
    rank = 32
    sigma = torch.arange(1, rank + 1, device="cuda").float() ** -0.5
    mix = torch.randn((rank, width), generator=g, device="cuda")
    mix *= sigma[:, None] / sigma.square().sum().sqrt()
    if outliers:
        at = torch.randint(0, width, (4,), generator=g, device="cuda")
        mean[at] *= 10
        mix[:, at] *= 10
    out = torch.empty((n, width), dtype=dtype, device="cuda")
    for a in range(0, n, 65536):
        m = min(65536, n - a)
        z = torch.randn((m, rank), generator=g, device="cuda")
        x = torch.randn((m, width), generator=g, device="cuda").mul_(0.1)
        out[a:a + m] = torch.addmm(mean, z, mix).add_(x)
    return out


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "append":
        n, width, streams = case["tokens"], case["width"], case["streams"]
        num_blocks = _blocks(n) + 16
        # rows of a fused projection: the streams side by side
        rows = _rows(g, n, width * streams, torch.bfloat16, False)
        s["ld"] = width * streams
        s["src"] = [rows[:, j * width:(j + 1) * width]
                    for j in range(streams)]
        s["cache"] = [torch.randn((num_blocks, BLOCK, width), generator=g,
                                  device="cuda").bfloat16()
                      for _ in range(streams)]
        ids = rng.permutation(num_blocks)[:_blocks(n)]
        t = np.arange(n)
        slots = ids[t // BLOCK] * BLOCK + t % BLOCK
        if n > 8:
            slots[-1] = -1           # a padded batch: no token there
        s["slots"] = torch.from_numpy(slots).cuda()
        s["num_blocks"] = num_blocks
        return s
    lens = rng.permutation(_lengths(case))
    n, longest = case["requests"], int(lens.max())
    max_blocks = max(1, int(_blocks(longest)))
    s["max_blocks"] = max_blocks
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    if case["op"] == "assign":
        held = np.maximum(lens - case["step"], 0) if case["step"] else 0 * lens
        before = _blocks(held)
        after = _blocks(lens)
        ids = rng.permutation(int(after.sum()) + 64).astype(np.int32)
        table = np.full((n, max_blocks), -1, np.int32)
        has = np.arange(max_blocks)[None, :] < before[:, None]
        table[has] = ids[:int(before.sum())]
        # blocks already given out stand before the head of the free list
        s["head"] = torch.tensor([int(before.sum())], device="cuda")
        s["free"] = torch.from_numpy(ids).cuda()
        s["held"] = torch.from_numpy(held.astype(np.int32)).cuda()
        s["table"] = torch.from_numpy(table).cuda()
        s["slots"] = torch.zeros(int((lens - held).sum()), dtype=torch.int64,
                                 device="cuda")
        s["cu"] = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
        s["held_out"] = torch.zeros_like(s["held"])
        s["head_out"] = torch.zeros_like(s["head"])
        return s
    heads, kv_heads, hd = case["heads"], case["kv_heads"], case["head_dim"]
    dtype = DTYPES[case["dtype"]]
    width = kv_heads * hd
    blocks = _blocks(lens)
    num_blocks = int(blocks.sum()) + 4
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((n, max_blocks), -1, np.int32)
    has = np.arange(max_blocks)[None, :] < blocks[:, None]
    table[has] = ids[:int(blocks.sum())]
    s["table"] = torch.from_numpy(table).cuda()
    s["num_blocks"] = num_blocks
    s["k"] = _rows(g, num_blocks * BLOCK, width, dtype, True).view(
        num_blocks, BLOCK, width)
    s["v"] = _rows(g, num_blocks * BLOCK, width, dtype, False).view(
        num_blocks, BLOCK, width)
    # the query heads of a fused projection's rows
    qkv = torch.randn((n, (heads + 2 * kv_heads) * hd), generator=g,
                      device="cuda").to(dtype)
    s["q"] = qkv[:, :heads * hd]
    s["q_ld"] = qkv.stride(0)
    s["scale"] = hd ** -0.5
    return s


# --------------------------------------------------------------- plain form
def _plain_assign(s):
    held, lens = s["held"].long(), s["lens"].long()
    room = s["max_blocks"] * BLOCK
    new = (lens - held).clamp_min(0)
    fits = lens <= room
    need = torch.where(fits & (new > 0), _blocks(lens) - _blocks(held), 0)
    total = need.cumsum(0)
    served = fits & ((need == 0) | (s["head"] + total <= s["free"].numel()))
    need = torch.where(served, need, 0)
    first = s["head"] + total - need
    cols = torch.arange(s["max_blocks"], device="cuda")[None, :]
    at = cols - _blocks(held)[:, None]
    fresh = (at >= 0) & (at < need[:, None])
    pick = (first[:, None] + at).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][pick], s["table"]))
    s["cu"][0] = 0
    s["cu"][1:] = new.cumsum(0)
    j = torch.arange(s["slots"].numel(), device="cuda")
    r = torch.searchsorted(s["cu"][1:], j, right=True)
    r = r.clamp_max(lens.numel() - 1)
    t = held[r] + j - s["cu"][r]
    ok = served[r] & (j < s["cu"][-1])
    b = s["table"][r, (t // BLOCK).clamp_max(s["max_blocks"] - 1)].long()
    s["slots"].copy_(torch.where(ok & (b >= 0), b * BLOCK + t % BLOCK, -1))
    s["held_out"].copy_(torch.where(served, torch.maximum(held, lens), held))
    s["head_out"].copy_(s["head"] + torch.where(need > 0, total, 0).amax())
    return _assign_outputs(s)


def _assign_outputs(s):
    return {"table": s["table"], "slots": s["slots"], "cu": s["cu"],
            "held": s["held_out"], "head": s["head_out"]}


def _plain_append(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    for rows, pool in zip(s["src"], s["cache"]):
        pool.view(-1, s["width"])[at] = rows[keep]
    return s["cache"]


def _plain_attend(s):
    n, kv_heads, hd = s["requests"], s["kv_heads"], s["head_dim"]
    group = s["heads"] // kv_heads
    length = s["max_blocks"] * BLOCK
    lens = s["lens"].long()[:, None]
    if s["window"]:
        sink, window = min(s["sink"], length), min(s["window"], length)
        t = torch.arange(-window, sink, device="cuda")[None, :]
        t = torch.where(t < 0, lens + t, t)
        recent = torch.arange(sink + window, device="cuda") < window
        valid = (t >= 0) & (t < lens) & ((t >= sink) | ~recent)
    else:
        t = torch.arange(length, device="cuda")[None, :].expand(n, length)
        valid = t < lens
    t = torch.where(valid, t, 0)
    row = s["table"].gather(1, t // BLOCK).long() * BLOCK + t % BLOCK
    row = torch.where(valid, row, 0)
    k = s["k"].view(-1, kv_heads, hd)[row].float()
    v = s["v"].view(-1, kv_heads, hd)[row].float()
    q = s["q"].float().reshape(n, kv_heads, group, hd)
    v = v.masked_fill(~valid[:, :, None, None], 0.0)
    x = torch.einsum("rhgd,rthd->rhgt", q, k) * s["scale"]
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("rhgt,rthd->rhgd", p, v) / torch.where(total == 0, 1.0,
                                                            total)
    lse = (m + torch.log(total)).view(n, s["heads"])
    return {"out": o.reshape(n, -1).to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------------------- run
def run(s):
    if not own:
        return {"assign": _plain_assign, "append": _plain_append,
                "attend": _plain_attend}[s["op"]](s)
    import kv_cache_transform_gb300 as kv
    if s["op"] == "append":
        kv.kvtc_paged_append(s["src"], s["ld"], s["tokens"], s["slots"],
                             s["width"], BLOCK, s["cache"], s["num_blocks"])
        return s["cache"]
    n = s["requests"]
    if s["op"] == "assign":
        if "workspace" not in s:
            size = kv.kvtc_paged_assign_workspace_bytes(n)
            s["workspace"] = torch.empty(size, dtype=torch.uint8,
                                         device="cuda")
        kv.kvtc_paged_assign(n, s["held"], s["lens"], s["free"],
                             s["free"].numel(), s["head"], s["table"],
                             s["max_blocks"], BLOCK, s["slots"],
                             s["slots"].numel(), s["cu"], s["held_out"],
                             s["head_out"], s["workspace"],
                             s["workspace"].numel())
        return _assign_outputs(s)
    heads, kv_heads, hd = s["heads"], s["kv_heads"], s["head_dim"]
    if "workspace" not in s:
        size = kv.kvtc_paged_attend_workspace_bytes(n, heads, kv_heads, hd)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty((n, heads * hd), dtype=s["q"].dtype, device="cuda")
    lse = torch.empty((n, heads), dtype=torch.float32, device="cuda")
    dtype = kv.KVTC_DTYPE_FP16 if s["dtype"] == "fp16" else kv.KVTC_DTYPE_BF16
    kv.kvtc_paged_attend(n, heads, kv_heads, hd, dtype, s["q"], s["q_ld"],
                         s["k"], s["v"], s["num_blocks"], BLOCK, s["table"],
                         s["max_blocks"], s["lens"], s["sink"], s["window"],
                         s["scale"], out, heads * hd, lse, s["workspace"],
                         s["workspace"].numel())
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    if case["op"] == "assign":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        source = np.full(s["num_blocks"] * BLOCK, -1)
        for i, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                source[at] = i
        source = torch.from_numpy(source).cuda()[:, None]
        return [torch.where(source >= 0, rows.double()[source.clamp_min(0)
                                                       [:, 0]],
                            pool.double().view(-1, s["width"]))
                .view(pool.shape) for rows, pool in zip(s["src"], s["cache"])]
    heads, kv_heads, hd = s["heads"], s["kv_heads"], s["head_dim"]
    out = torch.zeros((s["requests"], heads, hd), dtype=torch.float64,
                      device="cuda")
    lse = torch.full((s["requests"], heads), -math.inf, dtype=torch.float64,
                     device="cuda")
    group = heads // kv_heads
    for r, length in enumerate(s["lens"].tolist()):
        seen = [t for t in range(length) if not s["window"] or
                t < s["sink"] or t >= length - s["window"]]
        if not seen:
            continue
        seen = torch.tensor(seen, device="cuda")
        row = s["table"][r].long()[seen // BLOCK] * BLOCK + seen % BLOCK
        keys = s["k"].view(-1, kv_heads, hd)[row].double()
        values = s["v"].view(-1, kv_heads, hd)[row].double()
        queries = s["q"][r].double().view(heads, hd)
        for h in range(kv_heads):
            of = slice(h * group, (h + 1) * group)
            x = queries[of] @ keys[:, h].T * s["scale"]
            lse[r, of] = torch.logsumexp(x, 1)
            out[r, of] = torch.exp(x - lse[r, of][:, None]) @ values[:, h]
    return {"out": out.view(s["requests"], -1), "lse": lse}
