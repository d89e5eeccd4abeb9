"""Plain fp64 CPU oracle of causal attention with grouped heads, its gradient, and
the 8-bit key/value cache (test infrastructure only), one sequence at a time: q
[L_q, H_q, d], k, v [L_k, H_kv, d]; query i sees keys j <= i + L_k - L_q.

Bounds on what the kernels' arithmetic may differ by, element by element.  E is
the unit of the type that exp(s - max) and dS are rounded to before a product: half a
step of bf16, 2^-8, or 2^-22 for fp32 rows, whose three bf16 parts drop products
of 2^-24 of the largest and whose own parts end there.

Scores: a sum of d products in fp32 (at most d roundings of partial sums below
sum |q k|), times the scale: |ds| <= (d + 16) 2^-24 scale sum |q k|, and with fp32
rows three dropped products of 2^-24 more, which the 16 covers.  exp2's argument
is one fma of at most twice the largest score in log2 units, and the running
maximum times that: 4 2^-24 (|s| + |max|) more; exp2 itself is within 2^-22.  In
all a weight p is off by at most a relative e_s, the largest |ds| of its row plus
that.  o = sum p v / sum p: terms p |v| with 2 e_s (numerator and denominator), E, and
(L + 64) 2^-24 for the sums and rescalings.  lse: e_s, the logarithm's 2^-21 and
two roundings.

Gradient: p = exp(s - lse) is off by e_p = 2 e_s + that of lse; dP by (d + 16) 2^-24
sum |dO v|; dO . o by the same of sum |dO o| and by what o is off; dS = p (dP - D) by p
(e_p |dP - D| + those), and by E |dS| where it is rounded; dq, dk, dv are sums of
these times |k|, |q|, |dO| (p rounded by E for dv) with (L + 64) 2^-24 for the sums.

What lies below the smallest normal number, 2^-126 (fp32's and bf16's), may count as
0: a weight or a dS is off by that much besides, each time it enters a sum.
"""

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126


def _weights(q, k, scale):
    """Scores of every head [H_q, L_q, L_k] (-inf where not seen) and e_s [H_q, L_q]."""
    (lq, hq, d), (lk, hkv, _) = q.shape, k.shape
    g = hq // hkv
    kk = np.repeat(k, g, axis=1)
    s = scale * np.einsum("ihd,jhd->hij", q, kk)
    mag = scale * np.einsum("ihd,jhd->hij", np.abs(q), np.abs(kk))
    seen = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq
    s = np.where(seen, s, -np.inf)
    mag = np.where(seen, mag, 0.0)
    top = mag.max(axis=2) if lk else np.zeros((hq, lq))
    return s, (d + 16) * U * top + 8 * U * (1 + 1.5 * top) + 2.0 ** -22


def attn_fwd(q, k, v, scale, unit):
    """o [L_q, H_q, d], lse [L_q, H_q] and the bounds of both (without o's own rounding)."""
    (lq, hq, d), (lk, hkv, _) = q.shape, k.shape
    vv = np.repeat(v, hq // hkv, axis=1)
    s, es = _weights(q, k, scale)
    m = s.max(axis=2) if lk else np.full((hq, lq), -np.inf)
    some = np.isfinite(m)
    p = np.where(some[..., None], np.exp(s - np.where(some, m, 0.0)[..., None]), 0.0)
    z = p.sum(axis=2)
    with np.errstate(divide="ignore"):
        lse = np.where(some, np.where(some, m, 0.0) + np.log(z), -np.inf)
    p = p / np.where(some, z, 1.0)[..., None]
    o = np.einsum("hij,jhd->ihd", p, vv)
    mag = np.einsum("hij,jhd->ihd", p, np.abs(vv))
    bo = mag * (2 * es.T[..., None] + unit + (lk + 64) * U) + TINY * np.abs(vv).sum(axis=0)
    bl = np.where(some, es + 2.0 ** -21 + 4 * U * np.abs(np.where(some, lse, 0.0)), 0.0)
    return o, lse.T, bo, bl.T


def attn_bwd(q, k, v, do, scale, unit, half):
    """dict of (gradient, bound) for dq, dk, dv; half: o's own rounding."""
    (lq, hq, d), (lk, hkv, _) = q.shape, k.shape
    g = hq // hkv
    kk, vv = np.repeat(k, g, axis=1), np.repeat(v, g, axis=1)
    o, lse, bo, bl = attn_fwd(q, k, v, scale, unit)
    s, es = _weights(q, k, scale)
    some = np.isfinite(lse.T)
    p = np.where(some[..., None], np.exp(s - np.where(some, lse.T, 0.0)[..., None]), 0.0)
    dp = np.einsum("ihd,jhd->hij", do, vv)
    dd = np.einsum("ihd,ihd->hi", do, o)[..., None]
    ds = p * (dp - dd)
    ep = (2 * es + bl.T)[..., None]
    b_dp = (d + 16) * U * np.einsum("ihd,jhd->hij", np.abs(do), np.abs(vv))
    b_dd = ((d + 16) * U * np.einsum("ihd,ihd->hi", np.abs(do), np.abs(o)) +
            np.einsum("ihd,ihd->hi", np.abs(do), bo + half * (np.abs(o) + bo)))[..., None]
    b_ds = p * (1 + ep) * (ep * np.abs(dp - dd) + b_dp + b_dd)
    b_ds = b_ds + (unit + 4 * U) * (np.abs(ds) + b_ds) + TINY * (1 + np.abs(dp - dd)) * (s > -np.inf)
    n = (max(lq, lk) * g + 64) * U

    def fold(x):  # the heads of a group
        return x.reshape(lk, hkv, g, d).sum(axis=2)
    dq = scale * np.einsum("hij,jhd->ihd", ds, kk)
    bq = scale * np.einsum("hij,jhd->ihd", b_ds + n * np.abs(ds), np.abs(kk))
    dk = fold(scale * np.einsum("hij,ihd->jhd", ds, q))
    bk = fold(scale * np.einsum("hij,ihd->jhd", b_ds + n * np.abs(ds), np.abs(q)))
    dv = fold(np.einsum("hij,ihd->jhd", p, do))
    bv = fold(np.einsum("hij,ihd->jhd", p * (ep + unit + n) + TINY * (s > -np.inf), np.abs(do)))
    return {"dq": (dq, bq), "dk": (dk, bk), "dv": (dv, bv)}


# ---- the 8-bit cache ----------------------------------------------------------

BLOCK = 32


def e4m3_values():
    """The value of each of the 256 codes (fn: 0x7f and 0xff are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    x = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c >= 128, -x, x)


VALUES = e4m3_values()
_POS = VALUES[:127]  # increasing


def quantise(x, scale):
    """Codes of x / scale, to nearest, ties to the even code; not finite: NaN (0x7f, the sign aside)."""
    a = np.abs(np.where(np.isfinite(x), x, 0.0)) / scale
    cap = 240.0 if scale > 2.0 ** 119 else 448.0
    a = np.minimum(a, cap)
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isfinite(x), code, 127)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def scale_of(x):
    """The least power of two s >= 2^-117 with max |x| <= 448 s over the finite elements."""
    x = np.abs(np.where(np.isfinite(x), x, 0.0)).max() if x.size else 0.0
    s = 2.0 ** -117
    while x > 448 * s:
        s *= 2
    return s


class OracleCache:
    """Codes and scales [pages, H, ...] of keys or values, written block by block."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes.copy(), scales.astype(np.float64).copy()
        self.page_tokens = codes.shape[2]

    def write(self, x, table, start):
        """x [L, H, d] at the places start, start + 1, ... of one row of the block table."""
        t = start
        end = start + len(x)
        while t < end:
            b = t // BLOCK
            stop = min(end, (b + 1) * BLOCK)
            i, place = divmod(b * BLOCK, self.page_tokens)
            page = table[i] if i < len(table) else -1
            if 0 <= page < len(self.codes):
                for h in range(x.shape[1]):
                    s = scale_of(x[t - start:stop - start, h])
                    lo = t - b * BLOCK
                    if lo:
                        was = self.scales[page, h, place // BLOCK]
                        if was > s:
                            s = was
                        elif was < s:
                            old = VALUES[self.codes[page, h, place:place + lo]] * was
                            self.codes[page, h, place:place + lo] = quantise(old, s)
                    self.codes[page, h, place + lo:place + stop - b * BLOCK] = quantise(x[t - start:stop - start, h], s)
                    self.scales[page, h, place // BLOCK] = s
            t = stop

    def read(self, table, start, count):
        """Tokens [count, H, d]; NaN where no page holds them."""
        out = np.full((count, *self.codes.shape[1:2], self.codes.shape[3]), np.nan)
        there = np.zeros(count, bool)
        for t in range(start, start + count):
            i, place = divmod(t, self.page_tokens)
            page = table[i] if i < len(table) else -1
            if 0 <= page < len(self.codes):
                out[t - start] = VALUES[self.codes[page, :, place]] * self.scales[page, :, place // BLOCK][:, None]
                there[t - start] = True
        return out, there


def decode_fwd(q, k, v, there, scale, unit, kv_len):
    """Attention of q [L_q, H_q, d], the last of kv_len tokens, over those of k, v [n, ..]
    that a page holds: o, lse and their bounds."""
    lq, hq, d = q.shape
    o, lse = np.zeros((lq, hq, d)), np.full((lq, hq), -np.inf)
    bo, bl = np.zeros((lq, hq, d)), np.zeros((lq, hq))
    for i in range(lq):
        n = min(max(kv_len - lq + i + 1, 0), len(k))
        at = np.nonzero(there[:n])[0]
        if len(at) == 0:
            continue
        x = attn_fwd(q[i:i + 1], k[at], v[at], scale, unit)
        o[i], lse[i], bo[i], bl[i] = x[0][0], x[1][0], x[2][0], x[3][0]
    return o, lse, bo, bl
