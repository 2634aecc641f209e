"""Serving from a paged cache held in 4 bits on the GPU: the append with rotation,
the reading back and the attention, each against a plain fp64 implementation
(paged4_util.py, which derives the bounds), and a run of the three as a serving
loop makes it."""
import numpy as np
import pytest

import paged4_util as p4
import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int, host

pytestmark = pytest.mark.gpu

HEADS = [16, 32, 64, 128, 256]


def _bf16(rng, shape, std=1.0):
    return synthetic.round_to_bf16(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def _bytes(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# --------------------------------------------------------------------- append
def _append(rng, new, lens, h, h_kv, d, page, d_rot=0, interleaved=False, packed=False, k_exp=0, v_exp=-2, first=0,
            behind=0, base=10000.0, rows=None, in_place=False):
    """One append, checked against the definition: what the pages hold, the rows
    that they must not touch, and the rotated queries."""
    import torch
    cache = pu.Cache(rng, lens, h_kv, d, page)
    starts = pu.starts_of(new, first)
    t = int(starts[-1]) + behind
    q, k, v = (_bf16(rng, (t, n, d)) for n in (h, h_kv, h_kv)) if rows is None else rows
    dq, dk, dv = dev(q), dev(k), dev(v)
    if packed:
        both = torch.cat((dq, dk, dv), 1)
        dq, dk, dv = both[:, :h], both[:, h:h + h_kv], both[:, h + h_kv:]
    freqs = pu.freqs_of(d_rot, base)
    before = rng.integers(0, 256, (2, cache.n_pages, h_kv, page, 9 * d // 16)).astype(np.uint8)
    kp, vp = _bytes(before[0]), _bytes(before[1])
    q_out = dq if in_place else torch.full((t, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = sd.paged4_append(dq, dk, dv, kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens),
                           torch.from_numpy(freqs).cuda() if d_rot else None, interleaved, k_exp, v_exp, q_out)
    assert got.data_ptr() == q_out.data_ptr()
    sd.sdpa_device_check()
    pos = pu.positions_of(t, starts, lens)
    at = np.array([-1 if x is None else x for x in pos])
    ref_q, bound = pu.rotate(q, at, freqs, interleaved)
    out = host(q_out)
    for i in range(t):
        if pos[i] is None:
            assert np.all(out[i] == (q[i] if in_place else 7.0))
        else:
            assert np.all(np.abs(out[i] - ref_q[i]) <= bound[i] + 1e-30), i
    seq = np.searchsorted(starts, np.arange(t), side="right") - 1
    for pages, old, x, exp in ((kp, before[0], pu.rotate(k, at, freqs, interleaved)[0], k_exp),
                               (vp, before[1], v.astype(np.float64), v_exp)):
        want_codes, want_scales = p4.parts(old.copy(), d)
        codes, scales = p4.quantise(x, exp)
        for i in range(t):
            if pos[i] is None or pos[i] < 0:
                continue
            page_at = cache.table[seq[i], pos[i] // page]
            want_codes[page_at, :, pos[i] % page] = codes[i]
            want_scales[page_at, :, pos[i] % page] = scales[i]
        got_codes, got_scales = p4.parts(pages.cpu().numpy(), d)
        assert np.array_equal(got_scales, want_scales)
        # a zero's sign is not compared
        differ = (got_codes != want_codes) & ((got_codes & 7 != 0) | (want_codes & 7 != 0))
        assert not differ.any(), np.argwhere(differ)[:5]
    return cache, starts, kp, vp


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1, 1], [1, 129, 1000]), ([3, 0, 40, 1, 0], [17, 90, 40, 700, 0]),
                                      ([4, 1, 6], [2, 0, 6]), ([130], [130])])
def test_append_lengths(d, new, lens):
    rng = np.random.default_rng(1000 + d + sum(lens))
    _append(rng, new, lens, 4, 2, d, 16, d_rot=d // 2 // 16 * 16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,d_rot", [(d, r) for d in HEADS for r in sorted({0, 16, d // 2 // 16 * 16, d - 16, d}) if r <= d])
def test_append_rotations(d, d_rot, interleaved):
    rng = np.random.default_rng(1100 + d + d_rot + interleaved)
    _append(rng, [9, 1, 33], [40, 5000, 33], 6, 3, d, 32, d_rot=d_rot, interleaved=interleaved, packed=True)


@pytest.mark.parametrize("page", [16, 64, 512])
@pytest.mark.parametrize("k_exp,v_exp", [(0, 0), (-3, 4), (5, -9)])
def test_append_pages_and_units(page, k_exp, v_exp):
    rng = np.random.default_rng(1200 + page + k_exp)
    _append(rng, [2, 33, 1], [page - 1, 3 * page + 5, 777], 5, 1, 64, page, d_rot=64, k_exp=k_exp, v_exp=v_exp)


def test_append_leaves_other_rows_alone():
    rng = np.random.default_rng(1300)
    _append(rng, [3, 5], [100, 7], 4, 4, 32, 16, d_rot=32, first=4, behind=6)


def test_append_in_place_and_many_tokens():
    rng = np.random.default_rng(1301)
    _append(rng, [700, 1, 200], [700, 3000, 900], 4, 2, 64, 32, d_rot=64, in_place=True)


def test_append_many_blocks_against_the_definition():
    """Every code of 2700 tokens of 8 heads, far positions among them: blocks
    whose nearest scale or code fp32 leaves open are among these."""
    rng = np.random.default_rng(1302)
    _append(rng, [2000, 700], [2000, 150000], 8, 8, 128, 256, d_rot=128)


def test_append_borders():
    """Values halfway between two codes, blocks halfway between two scales,
    blocks whose scale is zero or the largest, zeros and infinities."""
    rng = np.random.default_rng(1303)
    d, t = 64, 64
    rows = np.zeros((t, 1, d), np.float32)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    for i in range(t):
        for b in range(4):
            s = np.float32(p4.E4M3[rng.integers(1, len(p4.E4M3))])
            x = rng.choice(np.concatenate((borders, [0.0, 6.0, 0.5, 4.0])), 16).astype(np.float32) * s
            x[rng.integers(16)] = 6 * s
            rows[i, 0, b * 16:(b + 1) * 16] = x * rng.choice(np.array([-1, 1], np.float32), 16)
    rows[1] = 0.0
    rows[2] = -0.0
    rows[3, 0, :16] = 6 * 2.0 ** -10       # between the scales 0 and 2^-9: zero
    rows[3, 0, 16:32] = 6.25 * 2.0 ** -10
    rows[4, 0, :16] = 1e30
    rows[4, 0, 20] = np.inf
    rows[5, 0, 3] = -np.inf
    for i in range(8, 40):                  # the largest element's sixth halfway between two scales
        lo = rng.integers(1, 125)
        rows[i, 0, :16] = 6 * (p4.E4M3[lo] + p4.E4M3[lo + 1]) / 2
    k = synthetic.round_to_bf16(rows)
    # (all of them bf16 numbers)
    assert np.array_equal(k[8:40], rows[8:40]) and np.array_equal(k[40:], rows[40:])
    q = _bf16(rng, (t, 1, d))
    _append(rng, [t], [t], 1, 1, d, 16, rows=(q, k, k.copy()), v_exp=0)
    _append(rng, [t], [t], 1, 1, d, 16, rows=(q, k, k.copy()), v_exp=0, packed=True)


def test_append_rotated_borders_at_position_zero():
    """Position 0 turns nothing: what lies on a border stays on it."""
    rng = np.random.default_rng(1304)
    d = 32
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0], np.float32)
    k = rng.choice(grid, (5, 4, d)).astype(np.float32) * rng.choice(np.array([-2, 1, 0.5], np.float32), (5, 4, d))
    _append(rng, [1] * 5, [1] * 5, 4, 4, d, 16, d_rot=32, rows=(k, k.copy(), k.copy()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,d_rot", [(64, 64), (128, 128), (256, 96), (16, 16)])
def test_append_angles_of_zero(d, d_rot, interleaved):
    """Pairs that do not turn (a frequency of zero), whole eights of them and some
    among others, at every position, and position 0: ties are as frequent as in
    rows that are not rotated at all."""
    import torch
    rng = np.random.default_rng(1901 + d)
    freqs = pu.freqs_of(d_rot)
    freqs[rng.random(len(freqs)) < 0.3] = 0.0
    freqs[len(freqs) // 2:] = 0.0
    n, h_kv, page = 70, 2, 32
    cache = pu.Cache(rng, [n], h_kv, d, page)
    # few significant bits: many elements on borders
    k = np.round(rng.standard_normal((n, h_kv, d)).astype(np.float32) * 4) / 4
    kp, vp = (torch.zeros((cache.n_pages, h_kv, page, 9 * d // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    sd.paged4_append(None, dev(k), dev(k), kp, vp, dev_int(cache.table), dev_int(pu.starts_of([n])), dev_int([n]),
                     torch.from_numpy(freqs).cuda(), interleaved=interleaved)
    sd.sdpa_device_check()
    for pages, x in ((kp, pu.rotate(k, np.arange(n), freqs, interleaved)[0]), (vp, k.astype(np.float64))):
        codes, scales = p4.quantise(x)
        got_codes, got_scales = p4.parts(pages.cpu().numpy(), d)
        for i in range(n):
            at = cache.table[0, i // page], slice(None), i % page
            assert np.array_equal(got_scales[at], scales[i])
            assert not ((got_codes[at] != codes[i]) & ((got_codes[at] & 7 != 0) | (codes[i] & 7 != 0))).any()


def _append_far(rng, k, last, freqs, interleaved):
    """Rows k as the last ones of a sequence of `last` positions, against a reference
    whose angles and functions are worked out in more than 64 bits."""
    import torch
    n, h_kv, d = k.shape
    page = 512
    table = np.full((1, last // page + 1), -1, np.int32)
    table[0, -2:] = 1, 0
    kp, vp = (torch.zeros((2, h_kv, page, 9 * d // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    sd.paged4_append(None, dev(k), dev(k), kp, vp, dev_int(table), dev_int(pu.starts_of([n])), dev_int([last]),
                     torch.from_numpy(freqs).cuda(), interleaved=interleaved)
    sd.sdpa_device_check()
    pos = np.arange(last - n, last)
    angle = pos.astype(np.longdouble)[:, None, None] * freqs.astype(np.longdouble)
    c, s = np.cos(angle), np.sin(angle)
    lo, hi = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    x = k.astype(np.longdouble)
    y = x.copy()
    y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., hi] * c + x[..., lo] * s
    codes, scales = p4.quantise(y.astype(np.float64))
    got_codes, got_scales = p4.parts(kp.cpu().numpy(), d)
    for i in range(n):
        at = table[0, pos[i] // page], slice(None), pos[i] % page
        assert np.array_equal(got_scales[at], scales[i])
        assert not ((got_codes[at] != codes[i]) & ((got_codes[at] & 7 != 0) | (codes[i] & 7 != 0))).any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("last", [(1 << 20) + 5, (1 << 29) - 3])
def test_append_at_far_positions(last, interleaved):
    rng = np.random.default_rng(1950 + interleaved)
    _append_far(rng, _bf16(rng, (300, 3, 64)), last, pu.freqs_of(64, 100.0), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pos", [491701844, 245850922, 710])
def test_append_next_to_whole_and_half_turns(pos, interleaved):
    """Angles that are a few 1e-9 (or 1e-5) beside a multiple of pi: elements on a border
    but for that."""
    rng = np.random.default_rng(1960 + interleaved)
    k = np.round(rng.standard_normal((1, 40, 64)).astype(np.float32) * 4) / 4
    _append_far(rng, k, pos + 1, np.ones(32, np.float32), interleaved)


def test_append_without_finite_rows_holds_finite_scales():
    import torch
    rng = np.random.default_rng(1305)
    cache = pu.Cache(rng, [9], 2, 64, 16)
    x = torch.full((9, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[3:] = float("inf")
    x[5, :, ::3] = 1.0
    kp, vp = (sd.paged4_pages(cache.n_pages, 2, 16, 64) for _ in range(2))
    args = (dev_int(cache.table), dev_int(pu.starts_of([9])), dev_int(cache.lens))
    sd.paged4_append(None, x, x, kp, vp, *args, torch.from_numpy(pu.freqs_of(64)).cuda())
    out = [torch.empty(9, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.paged4_read(kp, vp, *args, *out)
    assert all(bool(torch.isfinite(y).all()) for y in out)
    sd.sdpa_device_check()


# ----------------------------------------------------------------------- read
def _read(cache, pages, starts, t, exps=(0, 0), table=None):
    import torch
    out = [torch.full((t, cache.h_kv, cache.d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = sd.paged4_read(*pages, dev_int(cache.table if table is None else table), dev_int(starts),
                         dev_int(cache.lens), *out, *exps)
    assert got[0].data_ptr() == out[0].data_ptr() and got[1].data_ptr() == out[1].data_ptr()
    return [host(x) for x in out]


@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("d", HEADS)
def test_read_lengths(d, page):
    rng = np.random.default_rng(2000 + d + page)
    new, lens = [5, 0, 300, 1, 4], [90, 17, 300, 4000, 2]
    cache = pu.Cache(rng, lens, 3, d, page)
    starts = pu.starts_of(new, 2)
    t = int(starts[-1]) + 3
    dense = [[_bf16(rng, (n, 3, d), s) for n in lens] for s in (1.0, 0.1)]
    made = [p4.pages_of(cache, x, 0xFF, e) for x, e in zip(dense, (0, -5))]
    out = _read(cache, [_bytes(m[0]) for m in made], starts, t, (0, -5))
    pos = pu.positions_of(t, starts, lens)
    seq = np.searchsorted(starts, np.arange(t), side="right") - 1
    for got, (_, held) in zip(out, made):
        for i in range(t):
            if pos[i] is None:
                assert np.all(got[i] == 9.0)
            elif pos[i] < 0:
                assert np.all(got[i] == 0.0)
            else:
                assert np.array_equal(got[i], held[seq[i]][pos[i]])
    sd.sdpa_device_check()


def test_read_every_code_and_scale():
    """All 16 codes with all scales, in several units."""
    rng = np.random.default_rng(2100)
    d, page, n = 256, 16, 128
    cache = pu.Cache(rng, [n], 1, d, page)
    codes = np.broadcast_to(np.tile(np.arange(16), d // 16), (n, 1, d)).astype(np.int64)
    scales = (np.arange(n)[:, None, None] * np.ones((1, 1, d // 16), np.int64) % 127).astype(np.uint8)
    pages = np.zeros((cache.n_pages, 1, page * 9 * d // 16), np.uint8)
    packed = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
    for j in range(n):
        at, r = cache.table[0, j // page], j % page
        pages[at, :, r * d // 2:(r + 1) * d // 2] = packed[j]
        pages[at, :, page * d // 2 + r * d // 16:page * d // 2 + (r + 1) * d // 16] = scales[j]
    pages = _bytes(pages.reshape(cache.n_pages, 1, page, -1))
    for k_exp, v_exp in ((0, 0), (-32, 32), (7, -13)):
        k, v = _read(cache, (pages, pages), pu.starts_of([n]), n, (k_exp, v_exp))
        assert np.array_equal(k, p4.values(codes, scales, k_exp))
        assert np.array_equal(v, p4.values(codes, scales, v_exp))


# ------------------------------------------------------------------ attention
def _case(rng, new, lens, h, h_kv, d, page, fill=0xFF, std=1.0, first=0, behind=0, exps=(0, -3), window=0, sinks=0):
    """A cache whose unused rows hold bytes `fill` (0xFF: NaN scales), packed
    queries, and with a window tables without the pages that nobody sees."""
    cache = pu.Cache(rng, [max(n, 0) for n in lens], h_kv, d, page)
    cache.lens = np.asarray(lens, np.int32)
    if window:
        for s, (n, length) in enumerate(zip(new, lens)):
            start = max(0, length - n - window + 1)
            for x in range(-(-min(sinks, start) // page), start // page):
                cache.table[s, x] = -1 if x % 2 else cache.n_pages + 5
    table = cache.table.copy()
    cache.table = np.where(table >= cache.n_pages, -1, table)
    dense = [[_bf16(rng, (max(n, 0), h_kv, d), s) for n in lens] for s in (std, 0.3)]
    made = [p4.pages_of(cache, x, fill, e) for x, e in zip(dense, exps)]
    cache.table = table
    starts = pu.starts_of(new, first)
    q = _bf16(rng, (int(starts[-1]) + behind, h, d), std)
    return {"cache": cache, "pages": [m[0] for m in made], "held": [m[1] for m in made], "starts": starts, "q": q,
            "exps": exps, "window": window, "sinks": sinks}


def _args(c):
    return (dev(c["q"]), *(_bytes(x) for x in c["pages"]), dev_int(c["cache"].table), dev_int(c["starts"]),
            dev_int(c["cache"].lens))


def _kw(c):
    return {"k_exp": c["exps"][0], "v_exp": c["exps"][1], "window": c["window"], "sinks": c["sinks"]}


def _run(c, **kw):
    got = sd.paged4_attention(*_args(c), **dict(_kw(c), **kw))
    sd.sdpa_device_check()
    return got


def _check(got, c, scale=0.0):
    ref, bound = p4.attention(c["q"], *c["held"], c["starts"], np.maximum(c["cache"].lens, 0), scale, c["window"],
                              c["sinks"])
    got = host(got)
    rows = ~np.isnan(ref)
    assert np.all(np.isfinite(got[rows]))
    excess = np.abs(got - ref)[rows] - bound[rows]
    assert excess.max(initial=-1.0) <= 0, (excess.max(), np.abs(got - ref)[rows].max())


SEQS = [([1], [1]), ([1], [31]), ([1], [32]), ([1], [33]), ([1], [300]), ([5], [5]), ([130], [130]), ([70], [400]),
        ([1, 1, 1], [1, 129, 1000]), ([3, 0, 40, 1, 0], [17, 90, 40, 700, 0]), ([4, 1, 6], [2, 0, 6])]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("new,lens", SEQS)
def test_attention_lengths(d, new, lens):
    rng = np.random.default_rng(3000 + d + sum(new) + 7 * sum(lens))
    c = _case(rng, new, lens, 4, 2, d, 16)
    _check(_run(c), c)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("d", HEADS)
def test_attention_page_sizes(d, page):
    rng = np.random.default_rng(3100 + d + page)
    c = _case(rng, [2, 33, 1], [page - 1, 3 * page + 5, 777], 4, 2, d, page)
    _check(_run(c), c)


@pytest.mark.parametrize("h,h_kv", [(1, 1), (8, 8), (16, 4), (6, 2), (5, 1), (14, 2), (33, 1), (128, 1), (256, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_head_groups(d, h, h_kv):
    """Groups of whole tiles, and groups that a tile ends inside of."""
    rng = np.random.default_rng(3200 + d + h)
    c = _case(rng, [1, 7, 45], [200, 330, 45], h, h_kv, d, 32)
    _check(_run(c), c)


@pytest.mark.parametrize("d,h,h_kv,new,lens", [
    (128, 8, 1, [1], [20000]), (64, 4, 4, [1, 1, 1, 1], [5000, 3, 9000, 64]), (128, 4, 1, [96, 1], [4000, 7000]),
    (256, 2, 1, [3], [12000]), (128, 32, 1, [1], [20000]), (256, 16, 1, [2, 1], [9000, 5000]),
    (64, 33, 1, [1, 1], [9000, 4100]), (16, 8, 2, [4], [30000]), (32, 3, 1, [200], [3000]), (128, 1, 1, [1], [70000])])
def test_attention_split_walks(d, h, h_kv, new, lens):
    rng = np.random.default_rng(3300 + d + h)
    c = _case(rng, new, lens, h, h_kv, d, 64)
    _check(_run(c), c)


def test_attention_uneven_walks():
    rng = np.random.default_rng(3400)
    new = [700] + [1] * 12 + [90]
    lens = [700] + [int(x) for x in rng.integers(1500, 6000, size=12)] + [2500]
    c = _case(rng, new, lens, 16, 4, 64, 64)
    _check(_run(c), c)


@pytest.mark.parametrize("b,length,window,h,h_kv", [
    (28, 2000, 0, 8, 4), (28, 4000, 0, 8, 4), (100, 800, 0, 4, 4), (64, 1000, 0, 8, 4), (64, 2000, 0, 4, 4),
    (24, 3000, 1000, 8, 8), (48, 2000, 700, 4, 4), (4, 1000, 0, 16, 1), (33, 500, 0, 40, 2)])
def test_attention_cuts(b, length, window, h, h_kv):
    """Walks of about one length, of which there are just as many as the ways to cut
    them differ by, and lengths around them."""
    rng = np.random.default_rng(3450 + b + length)
    lens = [length + int(x) for x in rng.integers(-length // 3, length // 3, size=b)]
    c = _case(rng, [1] * b, lens, h, h_kv, 64, 64, window=window, sinks=4 if window else 0)
    _check(_run(c), c)
    lens = [length] * b
    c = _case(rng, [1] * b, lens, h, h_kv, 64, 64, window=window, sinks=4 if window else 0)
    _check(_run(c), c)


def test_attention_many_sequences():
    rng = np.random.default_rng(3401)
    lens = [int(x) for x in rng.integers(0, 200, size=600)]
    c = _case(rng, [1 if x % 7 else 0 for x in range(600)], lens, 2, 1, 32, 16)
    _check(_run(c), c)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (32, 128), (256, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (20, 3), (33, 64), (64, 0), (500, 100), (100000, 4), (40, 100000)])
def test_attention_windows(d, page, window, sinks):
    """Windows and sinks that end inside tiles and pages, pages of which nothing
    is visible named by entries that name no page, tokens before the window is full."""
    rng = np.random.default_rng(3500 + d + window + sinks)
    c = _case(rng, [1, 3, 60, 1, 2], [1, 700, 300, 1290, 1], 6, 2, d, page, window=window, sinks=sinks)
    _check(_run(c), c)


def test_attention_long_windows_split():
    rng = np.random.default_rng(3501)
    c = _case(rng, [1, 1, 4], [20000, 9000, 15000], 8, 1, 128, 64, window=6000, sinks=200)
    _check(_run(c), c)


def test_attention_scale_and_wide_range_of_queries():
    """Queries and scales that fp16 does not reach, rows of zeros."""
    rng = np.random.default_rng(3600)
    for exp, scale in ((100, 2.0 ** -101), (-100, 2.0 ** 90), (0, 0.3)):
        c = _case(rng, [3, 1], [50, 200], 4, 2, 64, 16)
        c["q"] = (c["q"] * np.float32(2.0 ** exp)).astype(np.float32)
        c["q"][1, 2] = 0.0
        _check(_run(c, scale=scale), c, scale)


def test_attention_rows_that_are_not_finite_stay_their_own():
    import torch
    rng = np.random.default_rng(3601)
    c = _case(rng, [2, 1], [50, 200], 4, 2, 64, 16)
    want = host(_run(c))
    c["q"][1, 2, 5] = np.nan
    c["q"][2, 0, 5] = np.inf
    got = host(_run(c))
    other = np.ones((3, 4), bool)
    other[1, 2] = other[2, 0] = False
    assert np.array_equal(got[other], want[other]) and np.isnan(got[1, 2]).all()


def test_attention_rows_of_no_sequence_stay():
    import torch
    rng = np.random.default_rng(3700)
    c = _case(rng, [3, 20], [100, 50], 4, 2, 64, 16, first=5, behind=4)
    out = torch.full((32, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    _check(_run(c, out=out), c)
    assert bool((out[:5] == 3.0).all()) and bool((out[28:] == 3.0).all())


def test_attention_strided_queries_and_streams():
    import torch
    rng = np.random.default_rng(3701)
    c = _case(rng, [3, 20], [1000, 50], 4, 2, 64, 16)
    args = list(_args(c))
    both = torch.zeros(23, 8, 64, dtype=torch.bfloat16, device="cuda")
    both[:, 2:6] = args[0]
    want = _run(c)
    args[0] = both[:, 2:6]
    got = sd.paged4_attention(*args, **_kw(c))
    assert torch.equal(got, want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = sd.paged4_attention(*args, **_kw(c), stream=stream)
    stream.synchronize()
    assert torch.equal(got, want)
    sd.sdpa_device_check()


def test_attention_repeats_bit_by_bit_whatever_the_workspace_holds():
    import torch
    rng = np.random.default_rng(3702)
    cases = [_case(rng, new, lens, h, h_kv, d, 32) for new, lens, h, h_kv, d in
             (([1], [40000], 8, 1, 128), ([40, 1], [300, 5000], 4, 2, 64), ([3], [9000], 2, 2, 256),
              ([130], [900], 6, 2, 32))]
    ready = [(_args(c), _kw(c)) for c in cases]
    want = [sd.paged4_attention(*a, **kw) for a, kw in ready]
    size = max(sd.paged4_workspace(a[0], a[1], a[3]).numel() for a, _ in ready)
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            for (args, kw), w in zip(ready, want):
                assert torch.equal(sd.paged4_attention(*args, **kw, workspace=ws), w)
    sd.sdpa_device_check()


def test_graphs_that_share_a_workspace_follow_their_lengths():
    import torch
    rng = np.random.default_rng(3703)
    c = _case(rng, [1, 1, 2], [9000, 500, 7000], 8, 2, 64, 64)
    args = _args(c)
    ws = sd.paged4_workspace(args[0], args[1], args[3])
    outs = [torch.zeros(4, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.paged4_attention(*args, **_kw(c), out=outs[0], workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sd.paged4_attention(*args, **_kw(c), out=out, workspace=ws)
        graphs.append(g)
    for lens in ([9000, 500, 7000], [8999, 2, 100], [1, 1, 2]):
        c["cache"].lens = np.asarray(lens, np.int32)
        args[5].copy_(dev_int(lens))
        for g, out in zip(graphs, outs):
            out.zero_()
            for _ in range(2):
                g.replay()
        held = [[x[:n] for x, n in zip(h, lens)] for h in c["held"]]
        for out in outs:
            _check(out, dict(c, held=held))
    sd.sdpa_device_check()


def test_bad_pages_are_reported_and_read_as_zeros():
    rng = np.random.default_rng(3704)
    for bad in (-1, 10 ** 6):
        c = _case(rng, [1, 2], [200, 90], 4, 2, 64, 16)
        starts, lens = c["starts"], c["cache"].lens
        c["cache"].table[0, 3] = bad
        for held in c["held"]:
            held[0][48:64] = 0.0
        got = sd.paged4_attention(*_args(c), **_kw(c))
        with pytest.raises(sd.SdpaError) as e:
            sd.sdpa_device_check()
        assert e.value.status == 7
        _check(got, c)
        pages = [_bytes(x) for x in c["pages"]]
        out = _read(c["cache"], pages, pu.starts_of([200, 0]), 200, c["exps"])
        with pytest.raises(sd.SdpaError):
            sd.sdpa_device_check()
        for x, held in zip(out, c["held"]):
            assert np.array_equal(x, held[0])
        k = dev(_bf16(rng, (1, 2, 64)))
        before = [x.clone() for x in pages]
        lengths = dev_int([50, 0])
        sd.paged4_append(None, k, k, *pages, dev_int(c["cache"].table), dev_int(pu.starts_of([1, 0])), lengths)
        with pytest.raises(sd.SdpaError):
            sd.sdpa_device_check()
        assert all(bool((x == y).all()) for x, y in zip(pages, before))


def test_pages_beyond_32_bits():
    """Pages 6 GB into the cache: appended, read and attended to."""
    import torch
    rng = np.random.default_rng(3705)
    d, page, h_kv, n = 128, 256, 8, 600
    n_pages = 6 * (1 << 30) // (h_kv * page * 72) + 1
    kp, vp = (torch.zeros((n_pages, h_kv, page, 72), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = dev_int(np.array([[n_pages - 1, n_pages - 3, n_pages - 2]], np.int32))
    k, v, q = (_bf16(rng, (n, x, d)) for x in (h_kv, h_kv, 16))
    starts, lens = dev_int(pu.starts_of([n])), dev_int([n])
    sd.paged4_append(None, dev(k), dev(v), kp, vp, table, starts, lens)
    out = [torch.empty(n, h_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.paged4_read(kp, vp, table, starts, lens, *out)
    held = [p4.values(*p4.quantise(x)) for x in (k, v)]
    assert all(np.array_equal(host(x), y) for x, y in zip(out, held))
    got = host(sd.paged4_attention(dev(q), kp, vp, table, starts, lens))
    ref, bound = p4.attention(q, [held[0]], [held[1]], pu.starts_of([n]), [n])
    assert np.all(np.abs(got - ref) <= bound)
    sd.sdpa_device_check()


def test_serving_loop():
    """A prompt, steps of single tokens and a draft, appended and attended to
    with a window; the cache read back stands for what was attended to."""
    import torch
    rng = np.random.default_rng(3800)
    h, h_kv, d, page, window, sinks = 8, 2, 64, 16, 100, 5
    freqs = pu.freqs_of(d)
    lens = np.zeros(3, np.int32)
    total = [300, 40, 170]
    cache = pu.Cache(rng, total, h_kv, d, page)
    kp, vp = (sd.paged4_pages(cache.n_pages, h_kv, page, d) for _ in range(2))
    table = dev_int(cache.table)
    held = [[np.zeros((0, h_kv, d)) for _ in range(3)] for _ in range(2)]
    for new in ([200, 30, 0], [1, 1, 150], [1, 0, 1], [4, 4, 4], [1, 1, 1]):
        lens = lens + np.asarray(new, np.int32)
        starts = pu.starts_of(new)
        t = int(starts[-1])
        q, k, v = _bf16(rng, (t, h, d)), _bf16(rng, (t, h_kv, d)), _bf16(rng, (t, h_kv, d), 0.3)
        rot = sd.paged4_append(dev(q), dev(k), dev(v), kp, vp, table, dev_int(starts), dev_int(lens),
                               torch.from_numpy(freqs).cuda(), v_exp=-3)
        out = sd.paged4_attention(rot, kp, vp, table, dev_int(starts), dev_int(lens), v_exp=-3, window=window,
                                  sinks=sinks)
        pos = np.array(pu.positions_of(t, starts, lens))
        kr = p4.values(*p4.quantise(pu.rotate(k, pos, freqs, False)[0]))
        vr = p4.values(*p4.quantise(v, -3), -3)
        for s in range(3):
            rows = slice(int(starts[s]), int(starts[s + 1]))
            held[0][s] = np.concatenate((held[0][s], kr[rows]))
            held[1][s] = np.concatenate((held[1][s], vr[rows]))
        ref, bound = p4.attention(host(rot), *held, starts, lens, 0.0, window, sinks)
        assert np.all(np.abs(host(out) - ref) <= bound)
    back = [torch.empty(int(lens.sum()), h_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.paged4_read(kp, vp, table, dev_int(pu.starts_of(lens)), dev_int(lens), *back, v_exp=-3)
    for x, y in zip(back, held):
        assert np.array_equal(host(x), np.concatenate(y))
    sd.sdpa_device_check()
