"""Cases of the operators around chunks of new tokens over paged caches: norms
and rotation of queries and keys with their way into the pools, attention of a
chunk, attention weight gathered per cached token, eviction by that weight.

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
def _rotate(name, tokens, heads, kv_heads, head_dim, dtype="bf16", rotary=0,
            interleaved=False, norm=False, factor=1.0):
    """rotary: rotated elements of a head (0: all); factor: how far the
    frequencies of long wavelengths are stretched."""
    return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
            "rotary": rotary or head_dim, "interleaved": interleaved,
            "norm": norm, "factor": factor}


def _chunks(name, requests, new_lo, new_hi, held_lo, held_hi, heads, kv_heads,
            head_dim, dtype="bf16", sink=0, window=0, pad=0):
    """new: tokens of the chunk, held: tokens in the cache before it."""
    return {"name": name, "op": "chunks", "requests": requests,
            "new_lo": new_lo, "new_hi": new_hi, "held_lo": held_lo,
            "held_hi": held_hi, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "sink": sink,
            "window": window, "pad": pad}


def _weigh(name, requests, rows, held_lo, held_hi, heads, kv_heads, head_dim,
           dtype="bf16", sink=0, window=0, decay=0.0):
    return {"name": name, "op": "weigh", "requests": requests,
            "new_lo": rows, "new_hi": rows, "held_lo": held_lo,
            "held_hi": held_hi, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "sink": sink,
            "window": window, "pad": 0, "decay": decay}


def _evict(name, requests, lo, hi, keep, sink, window, width, streams=2):
    return {"name": name, "op": "evict", "requests": requests, "lo": lo,
            "hi": hi, "keep": keep, "sink": sink, "window": window,
            "width": width, "streams": streams}


def listed():
    return [
        # one decode step of 64 requests, rotation alone
        _rotate("rotate_decode_64", 64, 28, 4, 128),
        # an 8192-token prompt, one layer: norms, stretched frequencies
        _rotate("rotate_prefill_8k", 8192, 32, 8, 128, norm=True, factor=8.0),
        # an odd number of tokens, a quarter of wide heads, neighbours paired
        _rotate("rotate_1000_part", 1000, 16, 2, 256, "fp16", rotary=64,
                interleaved=True),
        # the smallest chunk: 16 tokens behind 240, two heads; latency alone
        _chunks("chunk_tiny_16", 1, 16, 16, 240, 240, 2, 2, 64),
        # a whole 8192-token prompt, four query heads a KV head
        _chunks("chunk_prompt_8k", 1, 8192, 8192, 0, 0, 32, 8, 128),
        # 64 requests in one batch: decode steps, short and long chunks
        # behind ragged contexts, a padded batch, seven heads a KV head
        _chunks("chunk_64_ragged_g7", 64, 1, 256, 0, 3840, 28, 4, 128,
                pad=37),
        # the last 512 tokens of a long document
        _chunks("chunk_512_of_32k", 1, 512, 512, 32256, 32256, 32, 8, 128),
        # sink and window (the codec's 4 sink tokens), wide heads, fp16
        _chunks("chunk_window_8", 8, 100, 500, 1000, 8000, 16, 2, 256,
                "fp16", sink=4, window=1024),
        # weights of one decode step, added to what there is
        _weigh("weigh_decode_64", 64, 1, 0, 4095, 28, 4, 128, decay=1.0),
        # weights of a prompt's last 32 rows, eight heads a KV head
        _weigh("weigh_last_32", 16, 32, 968, 16352, 64, 8, 128),
        # a batch cut to 1024 tokens a request, K and V of one layer
        _evict("evict_64_to_1k", 64, 1, 4096, 1024, 4, 128, 512),
        # one long request cut to an eighth
        _evict("evict_32k_to_4k", 1, 32768, 32768, 4096, 4, 128, 1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "chunks", "chunks", "weigh", "evict"])
    head_dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
    heads = kv_heads * group
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rotate":
        most = max(1, min(16384, (40 << 20) // ((heads + 2 * kv_heads) *
                                                head_dim)))
        case = _rotate("", _log_int(rng, 1, most), heads, kv_heads, head_dim,
                       dtype, rng.choice([0, 0, head_dim // 2,
                                          8 * rng.randint(1, head_dim // 8)]),
                       rng.random() < 0.4, rng.random() < 0.5,
                       rng.choice([1.0, 4.0, 8.0]))
    elif op == "evict":
        hi = _log_int(rng, 1, 32768)
        width = 64 * _log_int(rng, 1, 32)
        most = max(1, min(256, (1 << 26) // (hi * width)))
        sink, window = rng.randint(0, 8), _log_int(rng, 1, 256)
        keep = sink + window + _log_int(rng, 1, 8192)
        case = _evict("", _log_int(rng, 1, most), rng.randint(0, hi), hi,
                      keep, sink, window, width, rng.choice([1, 2, 2, 4]))
    else:
        sink, window = rng.choice([(0, 0), (0, 0), (0, 0),
                                   (rng.randint(0, 40),
                                    _log_int(rng, 1, 4096))])
        held_hi = _log_int(rng, 1, 32768)
        held_lo = rng.randint(0, held_hi)
        if op == "weigh":
            rows = rng.choice([1, 1, _log_int(rng, 1, 64)])
            cost = rows * heads * head_dim * (held_hi + rows)
            cost = max(cost, 32 * kv_heads * head_dim * held_hi)
            most = max(1, min(128, (1 << 34) // cost))
            case = _weigh("", _log_int(rng, 1, most), rows, held_lo, held_hi,
                          heads, kv_heads, head_dim, dtype, sink, window,
                          rng.choice([0.0, 1.0, 0.9]))
        else:
            new_hi = _log_int(rng, 1, 4096)
            cost = new_hi * heads * head_dim * (held_hi + new_hi // 2 + 1)
            while cost > 1 << 37:
                new_hi //= 2
                cost = new_hi * heads * head_dim * (held_hi + new_hi // 2 + 1)
            cost = max(cost, 32 * kv_heads * head_dim * (held_hi + new_hi))
            most = max(1, min(128, (1 << 36) // cost))
            case = _chunks("", _log_int(rng, 1, most),
                           rng.randint(1, new_hi), new_hi, held_lo, held_hi,
                           heads, kv_heads, head_dim, dtype, sink, window,
                           rng.choice([0, 0, rng.randint(1, 50)]))
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n lengths spread evenly from lo to hi, so that their sum is the
    case's and not the seed's."""
    if n == 1:
        return np.array([hi], np.int64)
    return lo + (hi - lo) * np.arange(n, dtype=np.int64) // (n - 1)


def _chunk_lengths(case):
    """New tokens and lengths after the chunk; many new tokens come behind
    few held ones and the other way round."""
    new = _spread(case["requests"], case["new_lo"], case["new_hi"])
    held = _spread(case["requests"], case["held_lo"], case["held_hi"])
    if case["requests"] > 1:
        held = held[::-1]
    return new, held + new


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def work(case):
    if case["op"] == "rotate":
        n = case["tokens"]
        rows = n * (case["heads"] + 2 * case["kv_heads"]) * case["head_dim"]
        turned = n * (case["heads"] + case["kv_heads"])
        return {"bytes": 4 * rows + 12 * n + 4 * case["rotary"],
                "flops": turned * (3 * case["rotary"] + case["norm"] * 4 *
                                   case["head_dim"])}
    if case["op"] == "evict":
        lens = _spread(case["requests"], case["lo"], case["hi"])
        kept = np.minimum(lens, case["keep"])
        rows = int(kept.sum()) * case["width"] * case["streams"] * 2
        return {"bytes": 2 * rows + 4 * int(lens.sum()) + 8 * int(kept.sum())
                + 8 * case["requests"] +
                8 * int(_blocks(kept).sum()), "flops": 0}
    new, lens = _chunk_lengths(case)
    heads, hd = case["heads"], case["head_dim"]
    width = case["kv_heads"] * hd
    span = case["sink"] + case["window"] if case["window"] else 1 << 40
    pairs = read = 0
    for n, length in zip(new.tolist(), lens.tolist()):
        upto = min(max(span - (length - n), 0), n)   # rows that see all
        first = length - n + 1
        pairs += upto * first + upto * (upto - 1) // 2 + (n - upto) * span \
            if upto < n else n * first + n * (n - 1) // 2
        read += min(length, span + n - 1)
    total = int(new.sum())
    small = 12 * case["requests"] + 4 * (read // BLOCK + 1)
    if case["op"] == "weigh":
        sums = int(lens.sum()) * (8 if case["decay"] else 4)
        return {"bytes": 2 * read * width + 2 * total * heads * hd +
                4 * total * heads + sums + small,
                "flops": 2 * heads * hd * pairs}
    return {"bytes": 4 * read * width + 4 * total * heads * hd +
            4 * total * heads + small, "flops": 4 * heads * hd * pairs}


# ---------------------------------------------------------------- prepare
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


def _frequencies(rotary, factor, base=500000.0, context=8192):
    """Angle a position, of each pair: wavelengths up to a quarter of the
    context as they are, from the context on stretched by factor, between
    them a mixture."""
    f = base ** (-np.arange(0, rotary, 2) / rotary)
    turns = context * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
    return f * (keep + (1 - keep) / factor)


def _table(rng, lens, first, total, cols):
    """Blocks of the requests, anywhere in [first, first + total)."""
    blocks = _blocks(lens)
    ids = (first + rng.permutation(total)).astype(np.int32)
    table = np.full((len(lens), cols), -1, np.int32)
    has = np.arange(cols)[None, :] < blocks[:, None]
    table[has] = ids[:int(blocks.sum())]
    return table


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "rotate":
        return _prepare_rotate(s, rng, g)
    if case["op"] == "evict":
        return _prepare_evict(s, rng, g)
    heads, kv_heads, hd = case["heads"], case["kv_heads"], case["head_dim"]
    dtype = DTYPES[case["dtype"]]
    order = rng.permutation(case["requests"])
    new, lens = (x[order] for x in _chunk_lengths(case))
    blocks = int(_blocks(lens).sum())
    s["num_blocks"] = blocks + 4
    s["max_blocks"] = max(1, int(_blocks(lens).max()))
    table = _table(rng, lens, 0, s["num_blocks"], s["max_blocks"])
    # a scheduler knows the lengths; the calls read them on the device
    s["new_list"], s["len_list"] = new.tolist(), lens.tolist()
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).cuda()
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["table"] = torch.from_numpy(table).cuda()
    s["k"] = _rows(g, s["num_blocks"] * BLOCK, kv_heads * hd, dtype,
                   True).view(-1, BLOCK, kv_heads * hd)
    # the query heads of a fused projection's rows, padded behind the last
    s["rows"] = int(new.sum()) + case["pad"]
    qkv = torch.randn((s["rows"], (heads + 2 * kv_heads) * hd), generator=g,
                      device="cuda").to(dtype)
    s["q"], s["q_ld"] = qkv[:, :heads * hd], qkv.stride(0)
    s["scale"] = hd ** -0.5
    if case["op"] == "chunks":
        s["v"] = _rows(g, s["num_blocks"] * BLOCK, kv_heads * hd, dtype,
                       False).view(-1, BLOCK, kv_heads * hd)
        s["out"] = torch.zeros((s["rows"], heads * hd), dtype=dtype,
                               device="cuda")
        s["lse"] = torch.zeros((s["rows"], heads), device="cuda")
        return s
    # what the attention of the same rows returned beside its outputs
    s["lse"] = torch.zeros((s["rows"], heads), device="cuda")
    for r, j, rows, x in _scores(s, torch.float32):
        s["lse"][rows, j * s["group"]:(j + 1) * s["group"]] = torch.logsumexp(
            x, -1).view(-1, s["group"])
    s["acc_ld"] = s["max_blocks"] * BLOCK
    s["acc"] = torch.rand((case["requests"], s["acc_ld"]), generator=g,
                          device="cuda")
    s["acc_out"] = torch.zeros_like(s["acc"])
    return s


def _prepare_rotate(s, rng, g):
    n, heads, kv_heads, hd = (s[k] for k in ("tokens", "heads", "kv_heads",
                                             "head_dim"))
    dtype = DTYPES[s["dtype"]]
    rows = torch.randn((n, (heads + 2 * kv_heads) * hd), generator=g,
                       device="cuda").to(dtype)
    s["ld"], width = rows.stride(0), kv_heads * hd
    s["q"] = rows[:, :heads * hd]
    s["k"] = rows[:, heads * hd:heads * hd + width]
    s["v"] = rows[:, heads * hd + width:]
    s["q_out"] = torch.zeros((n, heads * hd), dtype=dtype, device="cuda")
    # a chunk somewhere in a long context
    first = int(rng.integers(0, 100000))
    s["positions"] = torch.arange(first, first + n, dtype=torch.int32,
                                  device="cuda")
    s["inv_freq"] = torch.from_numpy(_frequencies(s["rotary"],
                                                  s["factor"])).cuda()
    s["q_norm"] = s["k_norm"] = None
    if s["norm"]:
        s["q_norm"], s["k_norm"] = (
            (1 + 0.2 * torch.randn(hd, generator=g, device="cuda")).to(dtype)
            for _ in range(2))
    s["eps"] = 1e-6
    s["num_blocks"] = _blocks(n) + 8
    ids = rng.permutation(s["num_blocks"])[:_blocks(n)]
    t = np.arange(n)
    slots = ids[t // BLOCK] * BLOCK + t % BLOCK
    if n > 8:
        slots[-1] = -1           # a padded batch: no token there
    s["slots"] = torch.from_numpy(slots).cuda()
    s["pools"] = [torch.randn((s["num_blocks"], BLOCK, width), generator=g,
                              device="cuda").to(dtype) for _ in range(2)]
    return s


def _prepare_evict(s, rng, g):
    lens = rng.permutation(_spread(s["requests"], s["lo"], s["hi"]))
    kept = np.minimum(lens, s["keep"])
    before, after = int(_blocks(lens).sum()), int(_blocks(kept).sum())
    s["num_blocks"] = before + after + 4
    s["max_blocks"] = max(1, int(_blocks(lens).max()))
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    # the requests share their blocks with others: what is kept goes into
    # blocks of its own
    s["table"] = torch.from_numpy(_table(rng, lens, 0, before,
                                         s["max_blocks"])).cuda()
    s["out_table"] = torch.from_numpy(_table(rng, kept, before, after + 4,
                                             s["max_blocks"])).cuda()
    s["cache"] = [torch.randn((s["num_blocks"], BLOCK, s["width"]),
                              generator=g, device="cuda").bfloat16()
                  for _ in range(s["streams"])]
    # weights of attention: few large ones, many next to nothing
    s["acc_ld"] = s["max_blocks"] * BLOCK
    s["acc"] = torch.exp(3 * torch.randn((s["requests"], s["acc_ld"]),
                                         generator=g, device="cuda"))
    s["acc_out"] = torch.zeros_like(s["acc"])
    s["kept"] = torch.zeros((s["requests"], s["keep"]), dtype=torch.int32,
                            device="cuda")
    s["lens_out"] = torch.zeros_like(s["lens"])
    return s


# --------------------------------------------------------------- plain form
def _plain_rotate(s):
    hd, rd = s["head_dim"], s["rotary"]
    # (far positions: angles in 64 bits)
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    cos, sin = cos[:, None, :], sin[:, None, :]

    def turn(x, weight):
        x = x.float().reshape(x.shape[0], -1, hd)
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
            x = x * weight.float()
        y = x.clone()
        if s["interleaved"]:
            a, b = x[..., 0:rd:2], x[..., 1:rd:2]
            y[..., 0:rd:2] = a * cos - b * sin
            y[..., 1:rd:2] = b * cos + a * sin
        else:
            a, b = x[..., :rd // 2], x[..., rd // 2:rd]
            y[..., :rd // 2] = a * cos - b * sin
            y[..., rd // 2:rd] = b * cos + a * sin
        return y.reshape(x.shape[0], -1)

    s["q_out"].copy_(turn(s["q"], s["q_norm"]))
    k = turn(s["k"], s["k_norm"]).to(s["k"].dtype)
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    for rows, pool in zip((k, s["v"]), s["pools"]):
        pool.view(-1, rows.shape[1])[at] = rows[keep]
    return {"q": s["q_out"], "k": s["pools"][0], "v": s["pools"][1]}


def _scores(s, dtype):
    """Request, KV head, its rows, and their scores [rows * group][tokens],
    -inf where a row does not attend."""
    kv_heads, hd = s["kv_heads"], s["head_dim"]
    s["group"] = group = s["heads"] // kv_heads
    at = 0
    for r, (n, length) in enumerate(zip(s["new_list"], s["len_list"])):
        rows = slice(at, at + n)
        at += n
        t = torch.arange(length, device="cuda")
        place = s["table"][r].long()[t // BLOCK] * BLOCK + t % BLOCK
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        seen = t <= pos
        if s["window"]:
            seen &= (t < s["sink"]) | (t > pos - s["window"])
        hidden = ~seen.repeat_interleave(group, 0)
        keys = s["k"].view(-1, kv_heads, hd)[place]
        s["place"] = place
        for j in range(kv_heads):
            q = s["q"][rows, j * group * hd:(j + 1) * group * hd]
            x = q.to(dtype).reshape(n * group, hd) @ keys[:, j].to(dtype).T
            yield r, j, rows, x.mul_(s["scale"]).masked_fill_(hidden,
                                                              -math.inf)


def _plain_chunks(s):
    kv_heads, hd = s["kv_heads"], s["head_dim"]
    for r, j, rows, x in _scores(s, torch.float32):
        group = s["group"]
        m = x.amax(-1, keepdim=True)
        p = x.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        v = s["v"].view(-1, kv_heads, hd)[s["place"], j].float()
        o = (p @ v) / total
        s["out"][rows, j * group * hd:(j + 1) * group * hd] = o.view(
            -1, group * hd).to(s["out"].dtype)
        s["lse"][rows, j * group:(j + 1) * group] = (
            m + torch.log(total)).view(-1, group)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weigh(s):
    for r, j, rows, x in _scores(s, torch.float32):
        if j == 0:
            length = x.shape[1]
            to = s["acc_out"][r, :length]
            to.copy_(s["acc"][r, :length] * s["decay"])
        lse = s["lse"][rows, j * s["group"]:(j + 1) * s["group"]]
        to += torch.exp(x - lse.reshape(-1, 1)).sum(0)
    return s["acc_out"]


def _plain_evict(s):
    keep, cols = s["keep"], s["acc_ld"]
    lens = s["lens"].long()[:, None]
    t = torch.arange(cols, device="cuda")[None, :]
    rank = torch.where((t < s["sink"]) | (t >= lens - s["window"]), math.inf,
                       s["acc"])
    rank = torch.where(t < lens, rank, -1.0)
    # (stable: of equal ones the lowest index)
    first = torch.sort(rank, dim=1, descending=True, stable=True).indices
    first = torch.sort(first[:, :keep], dim=1).values
    n = first.shape[1]
    after = lens.clamp_max(keep)
    j = torch.arange(n, device="cuda")[None, :]
    has = j < after
    s["kept"].fill_(-1)
    s["kept"][:, :n] = torch.where(has, first, -1)
    s["lens_out"].copy_(after[:, 0])
    src = s["table"].gather(1, first // BLOCK).long() * BLOCK + first % BLOCK
    dst = s["out_table"].gather(1, (j // BLOCK).expand_as(first)).long()
    dst = dst * BLOCK + j % BLOCK
    for pool in s["cache"]:
        rows = pool.view(-1, s["width"])
        rows[dst[has]] = rows[src[has]]
    moved = torch.where(has, s["acc"].gather(1, first), 0.0)
    s["acc_out"].copy_(torch.where(t < lens, 0.0, s["acc_out"]))
    s["acc_out"][:, :n] = torch.where(has, moved, s["acc_out"][:, :n])
    return _evict_outputs(s)


def _evict_outputs(s):
    return {"kept": s["kept"], "lens": s["lens_out"], "acc": s["acc_out"],
            "cache": s["cache"]}


# --------------------------------------------------------------------- run
def run(s):
    if not own:
        return {"rotate": _plain_rotate, "chunks": _plain_chunks,
                "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)
    import kv_cache_transform_gb300 as kv
    if s["op"] == "evict":
        if "workspace" not in s:
            size = kv.kvtc_paged_evict_workspace_bytes(s["requests"],
                                                       s["max_blocks"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8,
                                         device="cuda")
        kv.kvtc_paged_evict(
            s["requests"], s["acc"], s["acc_ld"], s["lens"], s["keep"],
            s["sink"], s["window"], s["table"], s["out_table"],
            s["max_blocks"], BLOCK, s["cache"], s["width"], s["num_blocks"],
            s["kept"], s["acc_out"], s["lens_out"], s["workspace"],
            s["workspace"].numel())
        return _evict_outputs(s)
    heads, kv_heads, hd = s["heads"], s["kv_heads"], s["head_dim"]
    dtype = kv.KVTC_DTYPE_FP16 if s["dtype"] == "fp16" else kv.KVTC_DTYPE_BF16
    if s["op"] == "rotate":
        kv.kvtc_paged_rotate(
            s["tokens"], heads, kv_heads, hd, dtype, s["q"], s["k"], s["v"],
            s["ld"], s["positions"], s["inv_freq"], s["rotary"],
            s["interleaved"], 1.0, s["q_norm"], s["k_norm"], s["eps"],
            s["q_out"], s["q_out"].stride(0), s["slots"], BLOCK,
            s["pools"][0], s["pools"][1], s["num_blocks"])
        return {"q": s["q_out"], "k": s["pools"][0], "v": s["pools"][1]}
    if s["op"] == "weigh":
        if "workspace" not in s:
            size = kv.kvtc_paged_weigh_workspace_bytes(
                s["requests"], s["rows"], heads, kv_heads, hd)
            s["workspace"] = torch.empty(size, dtype=torch.uint8,
                                         device="cuda")
        kv.kvtc_paged_weigh(
            s["requests"], s["rows"], heads, kv_heads, hd, dtype, s["q"],
            s["q_ld"], s["k"], s["num_blocks"], BLOCK, s["table"],
            s["max_blocks"], s["cu"], s["lens"], s["sink"], s["window"],
            s["scale"], s["lse"], s["decay"], s["acc"], s["acc_out"],
            s["acc_ld"], s["workspace"], s["workspace"].numel())
        return s["acc_out"]
    if "workspace" not in s:
        size = kv.kvtc_paged_attend_chunks_workspace_bytes(
            s["requests"], s["rows"], heads, kv_heads, hd)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    kv.kvtc_paged_attend_chunks(
        s["requests"], s["rows"], heads, kv_heads, hd, dtype, s["q"],
        s["q_ld"], s["k"], s["v"], s["num_blocks"], BLOCK, s["table"],
        s["max_blocks"], s["cu"], s["lens"], s["sink"], s["window"],
        s["scale"], s["out"], heads * hd, s["lse"], s["workspace"],
        s["workspace"].numel())
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    kv_heads, hd = s["kv_heads"], s["head_dim"]
    group = s["heads"] // kv_heads
    chunks = case["op"] == "chunks"
    out = torch.zeros((s["rows"], s["heads"], hd), dtype=torch.float64,
                      device="cuda")
    lse = torch.zeros((s["rows"], s["heads"]), dtype=torch.float64,
                      device="cuda")
    acc = torch.zeros((case["requests"], s.get("acc_ld", 0)),
                      dtype=torch.float64, device="cuda")
    at = 0
    for r in range(case["requests"]):
        n, length = s["new_list"][r], s["len_list"][r]
        pool_rows = torch.tensor(
            [b * BLOCK + i for b in s["table"][r].tolist()
             for i in range(BLOCK)][:length], device="cuda")
        if not chunks and s["decay"]:
            acc[r, :length] = s["acc"][r, :length].double() * s["decay"]
        # a few rows at a time
        for i0 in range(0, n, 1024):
            m = min(1024, n - i0)
            end = length - n + i0 + m             # no row looks further
            pos = torch.arange(end - m, end, device="cuda")
            t = torch.arange(end, device="cuda")
            ahead = pos[:, None] - t[None, :]
            out_of = ahead < 0
            if s["window"]:
                out_of |= (ahead >= s["window"]) & (t >= s["sink"])[None, :]
            for h in range(s["heads"]):
                j = h // group
                of = slice(j * hd, (j + 1) * hd)
                keys = s["k"].view(-1, kv_heads * hd)[pool_rows[:end], of]
                q = s["q"][at + i0:at + i0 + m, h * hd:(h + 1) * hd].double()
                x = q @ keys.double().T * s["scale"]
                x[out_of] = -math.inf
                if chunks:
                    top = torch.logsumexp(x, 1)
                    lse[at + i0:at + i0 + m, h] = top
                    vals = s["v"].view(-1, kv_heads * hd)[pool_rows[:end], of]
                    out[at + i0:at + i0 + m, h] = torch.exp(
                        x - top[:, None]) @ vals.double()
                else:
                    top = s["lse"][at + i0:at + i0 + m, h].double()
                    acc[r, :end] += torch.exp(x - top[:, None]).sum(0)
        at += n
    if chunks:
        return {"out": out.view(s["rows"], -1), "lse": lse}
    return acc


def _exact_rotate(s):
    n, hd, rd = s["tokens"], s["head_dim"], s["rotary"]
    angle = torch.outer(s["positions"].double(), s["inv_freq"])
    factor = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turn(x, weight):
        x = x.double().reshape(n, -1, hd)
        if weight is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / hd +
                               s["eps"]) * weight.double()
        head = x[..., :rd]
        pairs = head.unflatten(-1, (rd // 2, 2)) if s["interleaved"] else \
            head.unflatten(-1, (2, rd // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(),
                                             pairs[..., 1].contiguous())
                               * factor)
        if not s["interleaved"]:
            z = z.transpose(-1, -2)
        return torch.cat([z.reshape(n, -1, rd), x[..., rd:]], -1).reshape(
            n, -1)

    source = np.full(s["num_blocks"] * BLOCK, -1)
    for i, at in enumerate(s["slots"].tolist()):
        if at >= 0:
            source[at] = i
    source = torch.from_numpy(source).cuda()

    def into(pool, rows):
        flat = pool.double().view(-1, rows.shape[1])
        return torch.where(source[:, None] >= 0, rows[source.clamp_min(0)],
                           flat).view(pool.shape)

    return {"q": turn(s["q"], s["q_norm"]),
            "k": into(s["pools"][0], turn(s["k"], s["k_norm"])),
            "v": into(s["pools"][1], s["v"].double())}


def _exact_evict(s):
    acc_out = s["acc_out"].double()
    cache = [pool.double() for pool in s["cache"]]
    table, out_table = s["table"].tolist(), s["out_table"].tolist()
    for r, length in enumerate(s["lens"].tolist()):
        weights = s["acc"][r].tolist()
        kept = list(range(length))
        if length > s["keep"]:
            free = range(s["sink"], length - s["window"])
            best = sorted(free, key=lambda t: (-weights[t], t))
            best = best[:s["keep"] - s["sink"] - s["window"]]
            kept = [*range(s["sink"]), *sorted(best),
                    *range(length - s["window"], length)]
        if not kept:
            continue
        acc_out[r, :length] = 0
        acc_out[r, :len(kept)] = s["acc"][r, kept].double()
        src = [table[r][t // BLOCK] * BLOCK + t % BLOCK for t in kept]
        dst = [out_table[r][j // BLOCK] * BLOCK + j % BLOCK
               for j in range(len(kept))]
        for pool in cache:
            rows = pool.view(-1, s["width"])
            rows[torch.tensor(dst, device="cuda")] = rows[
                torch.tensor(src, device="cuda")]
    return {"kept": None, "lens": None, "acc": acc_out, "cache": cache}
