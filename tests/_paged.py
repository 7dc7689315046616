"""Plain 64-bit forms of the paged serving calls, and their error bounds."""
import math

import numpy as np

BLOCK = 16


def blocks_of(tokens: int) -> int:
    return -(-tokens // BLOCK)


def assign(held, lens, free, head, table, slot_capacity):
    """kvtc_paged_assign from its definition, request by request.  Returns
    (table, slots, cu, held_out, head_out, short) with short true where the
    call reports KVTC_FLAG_SPACE."""
    table = np.array(table, np.int32)
    max_blocks = table.shape[1]
    head_ok = 0 <= head <= len(free)
    left = len(free) - head if head_ok else 0
    short = not head_ok
    cu, held_out, places = [0], [], []
    given = wanted = 0
    for r, (had, want) in enumerate(zip(held, lens)):
        had, want = max(int(had), 0), max(int(want), 0)
        new = max(want - had, 0)
        fits = want <= max_blocks * BLOCK
        need = blocks_of(want) - blocks_of(had) if new and fits else 0
        wanted += need
        served = fits and (need == 0 or wanted <= left)
        if served and need:
            for i in range(need):
                table[r, blocks_of(had) + i] = free[head + given + i]
            given += need
        short |= bool(new) and not served
        for t in range(had, want):
            b = int(table[r, t // BLOCK]) if served else -1
            places.append(b * BLOCK + t % BLOCK if b >= 0 else -1)
        cu.append(cu[-1] + new)
        held_out.append(max(had, want) if served else had)
    short |= len(places) > slot_capacity
    slots = np.full(slot_capacity, -1, np.int64)
    n = min(slot_capacity, len(places))
    slots[:n] = places[:n]
    return (table, slots, np.array(cu, np.int64),
            np.array(held_out, np.int32), head + given, short)


def attended(length, sink, window):
    """Positions that a request of `length` tokens attends to."""
    t = np.arange(max(length, 0))
    if window:
        t = t[(t < sink) | (t >= length - window)]
    return t


def attend(q, k, v, table, lens, sink, window, scale, unit):
    """Attention of one token per request in 64 bits.

    q [R][H][hd]; k, v [num_blocks][16][KV * hd] (float64); unit: half a step
    of the output type relative to the value.  Returns out, lse and bounds on
    how far a computation with 32-bit sums may be from them:

    a score is a sum of hd products scaled once: off by at most
    (hd + 2) 2^-23 scale sum|q k| (a tensor-core sum may truncate, one step
    of 2^-23 a term), and as an argument of exp2 by 2^-22 |s| more; a weight
    is then off by that (call it d, relative, doubled for exp(d) - 1 and the
    common maximum), by 2^-22 of exp2 and by 2^-16 for a weight that enters
    the product with v as two 16-bit parts; sums over n tokens add 2^-23 n.
    An output is off by the weighted mean of |v| times all that, on the
    weights and again on their sum, and by its own rounding."""
    R, H, hd = q.shape
    nb, _, width = k.shape
    KV = width // hd
    g = H // KV
    kf, vf = k.reshape(nb * BLOCK, KV, hd), v.reshape(nb * BLOCK, KV, hd)
    out, lse = np.zeros((R, H, hd)), np.full((R, H), -np.inf)
    tol_out, tol_lse = np.zeros((R, H, hd)), np.zeros((R, H))
    for r in range(R):
        length = min(max(int(lens[r]), 0), table.shape[1] * BLOCK)
        t = attended(length, sink, window)
        ids = table[r, t // BLOCK].astype(np.int64)
        ok = (ids >= 0) & (ids < nb)
        rows = ids[ok] * BLOCK + t[ok] % BLOCK
        n = len(rows)
        if n == 0:
            continue
        for j in range(KV):
            qs, ks, vs = q[r, j * g:(j + 1) * g], kf[rows, j], vf[rows, j]
            with np.errstate(all="ignore"):
                s = scale * (qs @ ks.T)
                m = s.max(1)
                base = np.where(m == -np.inf, 0.0, m)
                p = np.exp(s - base[:, None])
                l = p.sum(1)
                none = l == 0
                p = p / np.where(none, 1.0, l)[:, None]
                o = np.where(none[:, None], 0.0, p @ vs)
                ls = np.where(none, -np.inf, base + np.log(l))
                d = ((hd + 2) * 2.0 ** -23 * abs(scale) *
                     (np.abs(qs) @ np.abs(ks).T) + 2.0 ** -22 * np.abs(s))
                # tokens of no weight move nothing
                d = np.where(p > 1e-30, d, 0.0).max(1)
                e = 2 * d + 2.0 ** -21 + 2.0 ** -16 + n * 2.0 ** -23
                a = p @ np.abs(vs)
                to = (2 * e[:, None] * a + unit * np.abs(o) * (1 + 1e-6) +
                      2.0 ** -25)
                tl = d + (n + 8) * 2.0 ** -23 + 2.0 ** -22 * np.abs(ls)
            hs = slice(j * g, (j + 1) * g)
            out[r, hs], lse[r, hs] = o, ls
            tol_out[r, hs], tol_lse[r, hs] = to, tl
    return out, lse, tol_out, tol_lse


UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def check_attend(got_out, got_lse, ref):
    """Outputs (float64) against attend()'s, infinities and NaN in place."""
    out, lse, tol_out, tol_lse = ref
    for x, y, tol, what in ((got_out, out, tol_out, "out"),
                            (got_lse, lse, tol_lse, "lse")):
        if x is None:
            continue
        fine = np.isfinite(y)
        np.testing.assert_array_equal(np.isnan(x), np.isnan(y), what)
        np.testing.assert_array_equal(x[~fine & ~np.isnan(y)],
                                      y[~fine & ~np.isnan(y)], what)
        far = np.abs(x[fine] - y[fine]) - tol[fine]
        assert far.size == 0 or far.max() <= 0, (
            f"{what}: {int((far > 0).sum())} of {far.size} values further "
            f"off than the bound, worst by {far.max():.3g}")


def paged_case(seed, lens, heads, kv_heads, head_dim, extra_cols=1,
               spare_blocks=3, q_scale=1.0):
    """q, k, v pools, table: every block of a request in a shuffled place,
    rows that no request holds NaN, table columns behind a request's blocks
    far out of range.  float64 arrays of values that float16 and bfloat16
    both hold (seven bits)."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    R = len(lens)
    nb = np.array([blocks_of(max(int(n), 0)) for n in lens])
    cols = max(1, int(nb.max(initial=0)) + extra_cols)
    num_blocks = int(nb.sum()) + spare_blocks
    ids = rng.permutation(num_blocks)
    table = np.full((R, cols), 2 ** 31 - 1, np.int64)
    width = kv_heads * head_dim
    k = np.full((num_blocks, BLOCK, width), np.nan)
    v = np.full((num_blocks, BLOCK, width), np.nan)
    at = 0
    for r in range(R):
        table[r, :nb[r]] = ids[at:at + nb[r]]
        at += nb[r]
        n = max(int(lens[r]), 0)
        t = np.arange(n)
        rows = (table[r, t // BLOCK], t % BLOCK)
        k[rows] = bits7(rng.standard_normal((n, width)))
        v[rows] = bits7(rng.standard_normal((n, width)) + 0.5)
    q = bits7(rng.standard_normal((R, heads, head_dim)) * q_scale)
    return q, k, v, table.astype(np.int32), lens.astype(np.int32)


def bits7(x):
    """x rounded to seven significant bits (exact in bf16 and in fp16)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 128) / 128, np.maximum(e, -6))


def log_add(a, b):
    m = np.maximum(a, b)
    return m + np.log(np.exp(a - m) + np.exp(b - m))


def softmax_scale(head_dim):
    return 1.0 / math.sqrt(head_dim)
