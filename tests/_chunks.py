"""Plain 64-bit forms of the calls around chunks of new tokens, and their
error bounds."""
import fractions
import functools

import numpy as np

from _paged import BLOCK, UNIT, blocks_of

TWO_PI = fractions.Fraction(
    "6.283185307179586476925286766559005768394338798750211641949889")
STEP = 2.0 ** -23           # a step of fp32, relative


# ------------------------------------------------------------------ rotate
def rotate(x, weight, eps, positions, inv_freq, rotary_dim, interleaved,
           scale, unit):
    """x [N][heads][hd] (float64).  Returns y and a bound on how far a
    computation in fp32 may be from it: the norm's factor and each product
    are off by a few steps of fp32 (8 taken), the angle by 2^-25 of a turn,
    by a step of fp32 as an argument, and by p f 2^-52 through f / 2 pi in 64
    bits; then the output's own rounding."""
    x = x.astype(np.float64)
    if weight is not None:
        with np.errstate(all="ignore"):
            x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
    y, tol = x.copy(), 8 * STEP * np.abs(x)
    if rotary_dim:
        # (the angle modulo a turn, in whole numbers of 2^-64 turns)
        angle = np.empty((len(positions), len(inv_freq)))
        for i, p in enumerate(positions):
            for j, f in enumerate(inv_freq):
                angle[i, j] = turn_of(int(p), float(f))
        c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
        half = rotary_dim // 2
        ia, ib = ((slice(0, rotary_dim, 2), slice(1, rotary_dim, 2))
                  if interleaved else
                  (slice(0, half), slice(half, rotary_dim)))
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        off = (np.abs(a) + np.abs(b)) * abs(scale) * (
            16 * STEP + 2.0 ** -22 +
            np.abs(np.outer(positions, inv_freq))[:, None] * 2.0 ** -52)
        tol[..., ia] = tol[..., ib] = off
    return y, tol + unit * np.abs(y) * (1 + 1e-6) + 2.0 ** -26


@functools.lru_cache(maxsize=None)
def turns(f):
    """f / 2 pi in whole numbers of 2^-160 turns."""
    x = fractions.Fraction(f) / TWO_PI * 2 ** 160
    return round(x)


def turn_of(p, f):
    """p f modulo 2 pi, to 2^-120 or so."""
    at = p * turns(f) % 2 ** 160
    if at >= 2 ** 159:
        at -= 2 ** 160
    return at / 2 ** 160 * 6.283185307179586


# ----------------------------------------------------------------- chunks
def seen_by(pos, tokens, sink, window):
    """[rows][tokens]: which tokens the row at each position attends to."""
    t = np.arange(tokens)[None, :]
    pos = np.asarray(pos)[:, None]
    seen = t <= pos
    if window:
        seen &= (t < sink) | (t > pos - window)
    return seen


def chunk_rows(cu, lens, N, cols):
    """Per request: first row, rows, length (clamped as the calls do)."""
    out = []
    for r, length in enumerate(lens):
        c0, c1 = (min(max(int(c), 0), N) for c in cu[r:r + 2])
        out.append((c0, max(c1 - c0, 0),
                    min(max(int(length), 0), cols * BLOCK)))
    return out


def score_error(q, k, s, scale):
    """How far a score may be off in fp32, as in _paged.attend."""
    hd = q.shape[-1]
    return ((hd + 2) * STEP * abs(scale) * (np.abs(q) @ np.abs(k).T) +
            2.0 ** -22 * np.abs(s))


def attend_chunks(q, k, v, table, cu, lens, sink, window, scale, unit):
    """q [N][H][hd], k, v [num_blocks][16][KV * hd] float64.  out, lse (NaN
    rows where no request has them), and bounds as in _paged.attend, but for
    the weights' rounding: a weight enters the product with v as one 16-bit
    number (off by `unit`, relative, or in fp16 by 2^-32 of the largest weight
    where it is subnormal), its sum is of the unrounded ones."""
    N, H, hd = q.shape
    nb, _, width = k.shape
    KV = width // hd
    g = H // KV
    kf, vf = k.reshape(nb * BLOCK, KV, hd), v.reshape(nb * BLOCK, KV, hd)
    out, lse = np.full((N, H, hd), np.nan), np.full((N, H), np.nan)
    tol_out, tol_lse = np.zeros((N, H, hd)), np.zeros((N, H))
    has = np.zeros(N, bool)
    for r, (c0, n, length) in enumerate(chunk_rows(cu, lens, N,
                                                   table.shape[1])):
        if n == 0:
            continue
        rows = slice(c0, c0 + n)
        has[rows] = True
        t = np.arange(length)
        ids = table[r, t // BLOCK].astype(np.int64)
        ok = (ids >= 0) & (ids < nb)
        seen = seen_by(length - n + np.arange(n), length, sink, window)
        seen = seen[:, ok]
        at = ids[ok] * BLOCK + t[ok] % BLOCK
        for j in range(KV):
            ks, vs = kf[at, j], vf[at, j]
            for h in range(j * g, (j + 1) * g):
                qs = q[rows, h]
                with np.errstate(all="ignore"):
                    s = np.where(seen, scale * (qs @ ks.T), -np.inf)
                    m = s.max(1, initial=-np.inf)
                    base = np.where(m == -np.inf, 0.0, m)
                    p = np.where(seen, np.exp(s - base[:, None]), 0.0)
                    total = p.sum(1)
                    none = total == 0
                    p = p / np.where(none, 1.0, total)[:, None]
                    o = masked_product(p, vs, seen)
                    o = np.where(none[:, None], 0.0, o)
                    ls = np.where(none, -np.inf, base + np.log(total))
                    d = score_error(qs, ks, s, scale)
                    d = np.where(p > 1e-30, d, 0.0).max(1, initial=0.0)
                    count = seen.sum(1)
                    e = 2 * d + 2.0 ** -21 + count * STEP
                    a = masked_product(p, np.abs(vs), seen)
                    top = np.abs(np.where(np.isfinite(vs), vs, 0)).max(
                        initial=0.0)
                    to = ((2 * e + unit * (1 + 2 * e))[:, None] * a +
                          unit * np.abs(o) * (1 + 1e-2) + 2.0 ** -25 +
                          (count * 2.0 ** -31 * top)[:, None])
                    tl = d + (count + 8) * STEP + 2.0 ** -22 * np.abs(ls)
                out[rows, h], lse[rows, h] = o, ls
                tol_out[rows, h], tol_lse[rows, h] = to, tl
    return out, lse, tol_out, tol_lse, has


def masked_product(p, v, seen):
    """p @ v over the seen tokens alone (an infinite or NaN value counts for
    the rows that attend to it)."""
    fine = np.where(np.isfinite(v), v, 0.0)
    o = p @ fine
    odd = np.nonzero(~np.isfinite(v).all(1))[0]
    for t in odd:
        who = seen[:, t]
        extra = np.where(np.isfinite(v[t]), 0.0, v[t])
        with np.errstate(all="ignore"):
            add = np.where(np.isfinite(v[t])[None, :], 0.0,
                           p[who, t][:, None] * extra[None, :])
        o[who] += add
    return o


def check_chunks(got_out, got_lse, ref):
    out, lse, tol_out, tol_lse, has = ref
    for x, y, tol, what in ((got_out, out, tol_out, "out"),
                            (got_lse, lse, tol_lse, "lse")):
        if x is None:
            continue
        x, y, tol = x[has], y[has], tol[has]
        fine = np.isfinite(y)
        np.testing.assert_array_equal(np.isnan(x), np.isnan(y), what)
        np.testing.assert_array_equal(x[~fine & ~np.isnan(y)],
                                      y[~fine & ~np.isnan(y)], what)
        far = np.abs(x[fine] - y[fine]) - tol[fine]
        assert far.size == 0 or far.max() <= 0, (
            f"{what}: {int((far > 0).sum())} of {far.size} values further "
            f"off than the bound, worst by {far.max():.3g}")


# ------------------------------------------------------------------ weigh
def weigh(q, k, table, cu, lens, sink, window, scale, lse, decay, acc):
    """acc_out, with acc's own elements from lens on, and a bound: each
    weight is off by its exponent's error (the score's, and 2^-22 of |lse|),
    the sum of n of them by n steps of fp32."""
    N, H, hd = q.shape
    nb, _, width = k.shape
    KV = width // hd
    g = H // KV
    kf = k.reshape(nb * BLOCK, KV, hd)
    out, tol = acc.astype(np.float64).copy(), np.zeros(acc.shape)
    for r, (c0, n, length) in enumerate(chunk_rows(cu, lens, N,
                                                   table.shape[1])):
        rows = slice(c0, c0 + n)
        t = np.arange(length)
        ids = table[r, t // BLOCK].astype(np.int64)
        ok = (ids >= 0) & (ids < nb)
        seen = seen_by(length - n + np.arange(n), length, sink, window)
        seen = seen[:, ok]
        at = ids[ok] * BLOCK + t[ok] % BLOCK
        total, off = np.zeros(length), np.zeros(length)
        for h in range(H):
            ks, qs = kf[at, h // g], q[rows, h]
            with np.errstate(all="ignore"):
                s = scale * (qs @ ks.T)
                ls = lse[rows, h].astype(np.float64)[:, None]
                w = np.where(seen & (ls > -np.inf), np.exp(s - ls), 0.0)
                w = np.where(seen & np.isnan(ls), np.nan, w)
                d = score_error(qs, ks, s, scale) + 2.0 ** -22 * np.abs(
                    np.where(np.isfinite(ls), ls, 0))
                d = np.where(seen & (w > 1e-30), d, 0.0)
            total[ok] += w.sum(0)
            off[ok] += (w * (2 * d + 2.0 ** -21)).sum(0)
        start = acc[r, :length] * decay if decay else np.zeros(length)
        out[r, :length] = start + total
        tol[r, :length] = (off + (n * H + 4) * STEP *
                           (total + np.abs(start)) + 1e-30)
    return out, tol


# ------------------------------------------------------------------ evict
def evict(acc, lens, keep, sink, window, table, out_table, pools, in_place):
    """kept, acc_out, lens_out, pools (numpy, any dtype), and whether a block
    id was out of range, request by request."""
    kept_out = np.full((len(lens), keep), -1, np.int32)
    acc_out, after = acc.copy(), []
    new = [p.copy() for p in pools]
    nb = pools[0].shape[0] if pools else 1 << 31
    bad = False
    for r, length in enumerate(lens):
        length = min(max(int(length), 0), table.shape[1] * BLOCK)
        kept = list(range(length))
        if length > keep:
            w = np.where(np.isnan(acc[r]), -np.inf, acc[r])
            below = np.isnan(acc[r])
            free = range(sink, length - window)
            best = sorted(free, key=lambda t: (below[t], -w[t], t))
            best = sorted(best[:keep - sink - window])
            kept = [*range(sink), *best, *range(length - window, length)]
        after.append(len(kept))
        kept_out[r, :len(kept)] = kept
        moved = acc[r, kept]
        acc_out[r, :length] = 0
        acc_out[r, :len(kept)] = moved
        for j, t in enumerate(kept):
            a, b = int(table[r, t // BLOCK]), int(out_table[r, j // BLOCK])
            if not (0 <= a < nb and 0 <= b < nb):
                bad = True
                continue
            for p, o in zip(pools, new):
                o[b, j % BLOCK] = p[a, t % BLOCK]
    return kept_out, acc_out, np.array(after, np.int32), new, bad


__all__ = ["BLOCK", "UNIT", "blocks_of"]
