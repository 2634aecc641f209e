"""A plain fp64 implementation of the paged cache held in 4 bits, and the bounds
its GPU counterpart is held to.

What the cache holds is compared byte by byte (but for the sign of a zero):
scales and codes are nearest ones of exactly rounded quotients.

Bound of attention: o = sum_j w_j v_j over what the codes stand for, which is
exact in fp16.  The weights p_j are rounded to fp16 before the products (half a
step: 2^-11 of p_j, or 2^-25 where p_j is below 2^-14; p_j is relative to a
running maximum that no final one is below, so that the weights' sum is at least
1), o to bf16 after (2^-8).  The scores are sums of d products in fp32, off by at
most e = d 2^-23 scale sum_c |q_c k_c| (half of fp32's rounding allows for
accumulators that truncate, and for the elements of q below 2^-27 of the row's
largest), which moves a weight and the weights' sum by a factor exp(2 e)
together; the exponent (|x| <= 2^7 in fp32), ex2.approx and the fp32 sums of up
to 2^17 terms in a tree add at most 2^-14:
  (2^-11 + 2.1 e + 2^-14) sum_j w_j |v_j| + 2^-25 sum_j |v_j| + 2^-8 |o|, times 1 + 2^-8.
"""
import numpy as np

import paged_util as pu

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite e4m3 number from zero on, by its byte
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])


def _nearest(x, grid):
    """Index of the element of the increasing grid nearest to x >= 0; of two as
    near, the even one; of infinity the last."""
    x = np.minimum(x, 2 * grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, exp=0):
    """(codes, scales) of rows x [..., d]: 0 .. 15 [..., d] and bytes [..., d / 16]."""
    x = np.asarray(x, np.float64) * 2.0 ** -exp
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    scales = _nearest(np.abs(b).max(-1) / 6, E4M3)
    s = E4M3[scales][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(b) / s, 0.0)
    codes = _nearest(y, GRID) | np.where(b < 0, 8, 0)
    return codes.reshape(x.shape), scales.astype(np.uint8)


def values(codes, scales, exp=0):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(E4M3[scales], 16, -1) * 2.0 ** exp


def pages_of(cache, dense, fill=0xFF, exp=0):
    """Pages that hold `dense` (a list of [len, h_kv, d] arrays) quantised, and
    what they stand for (another such list); bytes `fill` everywhere else."""
    d, page = cache.d, cache.page
    out = np.full((cache.n_pages, cache.h_kv, page * 9 * d // 16), fill, np.uint8)
    held = []
    for s, x in enumerate(dense):
        codes, scales = quantise(x, exp)
        held.append(values(codes, scales, exp))
        packed = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
        for j in range(len(x)):
            at, r = cache.table[s, j // page], j % page
            if at < 0:
                continue
            out[at, :, r * d // 2:(r + 1) * d // 2] = packed[j]
            out[at, :, page * d // 2 + r * d // 16:page * d // 2 + (r + 1) * d // 16] = scales[j]
    return out.reshape(cache.n_pages, cache.h_kv, page, 9 * d // 16), held


def parts(pages, d):
    """(codes 0 .. 15 [n, h_kv, page, d], scales [n, h_kv, page, d / 16]) of pages' bytes."""
    n, h_kv, page, _ = pages.shape
    flat = pages.reshape(n, h_kv, -1)
    packed = flat[..., :page * d // 2].reshape(n, h_kv, page, d // 2)
    codes = np.stack((packed & 15, packed >> 4), -1).reshape(n, h_kv, page, d)
    return codes, flat[..., page * d // 2:].reshape(n, h_kv, page, d // 16)


def attention(q, dense_k, dense_v, starts, lens, scale=0.0, window=0, sinks=0):
    """(out, bound) for q [t, h, d] and what each sequence's cache stands for
    [len, h_kv, d]; rows of no sequence are NaN in `out`."""
    t, h, d = q.shape
    sc = scale if scale > 0 else 1.0 / np.sqrt(d)
    out = np.full((t, h, d), np.nan)
    bound = np.zeros((t, h, d))
    for s in range(len(lens)):
        a, e, length = int(starts[s]), int(starts[s + 1]), int(lens[s])
        k, v = dense_k[s], dense_v[s]
        h_kv = k.shape[1]
        for i in range(a, e):
            pos = length - e + i
            if pos < 0:
                out[i] = 0.0
                continue
            j = np.arange(pos + 1)
            if window:
                j = j[(j > pos - window) | (j < sinks)]
            kk, vv = k[j], v[j]
            qq = q[i].astype(np.float64).reshape(h_kv, h // h_kv, d)
            z = sc * np.einsum("ygd,jyd->ygj", qq, kk)
            w = np.exp(z - z.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            o = np.einsum("ygj,jyd->ygd", w, vv)
            err = d * 2.0 ** -23 * sc * np.einsum("ygd,jyd->ygj", np.abs(qq), np.abs(kk)).max(-1)[..., None]
            mass = np.einsum("ygj,jyd->ygd", w, np.abs(vv))
            total = np.abs(vv).sum(0)[:, None]
            out[i] = o.reshape(h, d)
            bound[i] = (((2.0 ** -11 + 2.1 * err + 2.0 ** -14) * mass + 2.0 ** -25 * total + 2.0 ** -8 * np.abs(o))
                        * (1 + 2.0 ** -8)).reshape(h, d)
    return out, bound


def rotate(x, positions, freqs, interleaved):
    return pu.rotate(x, positions, freqs, interleaved)[0]
