"""A plain fp64 implementation of serving from a paged cache, and the bounds
its GPU counterpart is held to.

Bounds (a bf16 rounding is off by at most 2^-8 of the value):
  append: the exact rotation of bf16 values, rounded once.  cos and sin are
    good to 2e-6 (the angle to 2^-22 of a turn = 1.5e-6 rad, and fp32's 2^-24
    in the function), the two products and their sum add 2^-23 of |a| + |b|:
      2^-8 |x| + 2.2e-6 (|a| + |b|), the second term rounded along: times 1 + 2^-8.
    Columns that are not rotated, and values, are copied: equal.
  attention: o = sum_j p_j v_j with p rounded to bf16 before the products and
    o rounded after: 2^-8 sum_j p_j |v_j| + 2^-8 |o|.  The scores are sums of d
    products in fp32, off by at most e = d 2^-23 scale sum_c |q_c k_c|
    (half of fp32's rounding allows for accumulators that truncate), which
    moves a weight and the weights' sum by a factor exp(2 e) together; the
    exponent (|x| <= 2^7 in fp32), ex2.approx and the fp32 sums of up to 2^17
    terms in a tree add at most 2^-14:
      (2^-8 + 2.1 e + 2^-14) sum_j p_j |v_j| + 2^-8 |o|, times 1 + 2^-8.
"""
import numpy as np


class Cache:
    """A paged cache with the bookkeeping of `lens` positions a sequence:
    shuffled pages, entries that no position needs left at -1."""

    def __init__(self, rng, lens, h_kv, d, page, spare=2, extra_columns=1):
        self.lens = np.asarray(lens, np.int32)
        self.h_kv, self.d, self.page = h_kv, d, page
        need = [-(-int(max(n, 0)) // page) for n in lens]
        self.n_pages = sum(need) + spare
        self.per_seq = max(max(need), 1) + extra_columns
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), self.per_seq), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n

    def pages_of(self, dense, fill):
        """Pages that hold `dense` (a list of [len, h_kv, d] arrays); `fill`
        everywhere else."""
        out = np.full((self.n_pages, self.h_kv, self.page, self.d), fill, np.float32)
        for s, x in enumerate(dense):
            for j in range(len(x)):
                out[self.table[s, j // self.page], :, j % self.page] = x[j]
        return out


def starts_of(new, first=0):
    return np.concatenate([[first], first + np.cumsum(new)]).astype(np.int32)


def attention(q, dense_k, dense_v, starts, lens, scale=0.0):
    """(out, bound) for q [t, h, d] and per-sequence keys and values
    [len, h_kv, d]; rows of no sequence are NaN in `out`."""
    t, h, d = q.shape
    sc = scale if scale > 0 else 1.0 / np.sqrt(d)
    out = np.full((t, h, d), np.nan)
    bound = np.zeros((t, h, d))
    for s in range(len(lens)):
        a, e, length = int(starts[s]), int(starts[s + 1]), int(lens[s])
        k, v = dense_k[s].astype(np.float64), dense_v[s].astype(np.float64)
        group = h // k.shape[1] if k.ndim == 3 and k.shape[1] else h
        for i in range(a, e):
            pos = length - e + i
            for x in range(h):
                if pos < 0:
                    out[i, x] = 0.0
                    continue
                kk, vv = k[:pos + 1, x // group], v[:pos + 1, x // group]
                qq = q[i, x].astype(np.float64)
                z = sc * (kk @ qq)
                w = np.exp(z - z.max())
                w /= w.sum()
                out[i, x] = w @ vv
                err = d * 2.0 ** -23 * sc * (np.abs(kk) @ np.abs(qq)).max()
                mass = w @ np.abs(vv)
                bound[i, x] = ((2.0 ** -8 + 2.1 * err + 2.0 ** -14) * mass + 2.0 ** -8 * np.abs(out[i, x])) * (1 + 2.0 ** -8)
    return out, bound


def rotate(x, positions, freqs, interleaved):
    """(rotated, bound) of rows x [t, heads, d] at the given positions."""
    x = x.astype(np.float64)
    out, bound = x.copy(), np.zeros_like(x)
    n = len(freqs)
    if n == 0:
        return out, bound
    angle = positions.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    c, s = np.cos(angle), np.sin(angle)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., lo], x[..., hi]
    out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
    slack = 2.2e-6 * (np.abs(a) + np.abs(b))
    for part in (lo, hi):
        bound[..., part] = (2.0 ** -8 * np.abs(out[..., part]) + slack) * (1 + 2.0 ** -8)
    return out, bound


def positions_of(t, starts, lens):
    """Position of every packed row; None for rows of no sequence."""
    out = [None] * t
    for s in range(len(lens)):
        for i in range(int(starts[s]), int(starts[s + 1])):
            out[i] = int(lens[s]) - int(starts[s + 1]) + i
    return out


def freqs_of(d_rot, base=10000.0):
    i = np.arange(0, d_rot, 2, dtype=np.float64)
    return (base ** (-i / max(d_rot, 1))).astype(np.float32)
