"""Serving from a paged cache on the GPU: the append with rotation and the
attention of packed new tokens, each against a plain fp64 implementation
(paged_util.py, which derives the bounds), and a run of the two as a serving
loop makes it."""
import numpy as np
import pytest

import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int, host

pytestmark = pytest.mark.gpu


def _bf16(rng, shape, std=1.0):
    return synthetic.round_to_bf16(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def _raw(x):
    """A tensor's bits, so that NaN compares."""
    import torch
    return x.contiguous().view(torch.int16)


# ------------------------------------------------------------------ attention
def _case(rng, new, lens, h, h_kv, d, page, fill=np.nan, std=1.0, first=0, behind=0):
    """A cache whose unused rows hold `fill`, packed queries (with `first`
    rows before and `behind` rows after those of the sequences)."""
    cache = pu.Cache(rng, lens, h_kv, d, page)
    dense = [[_bf16(rng, (max(n, 0), h_kv, d), s) for n in lens] for s in (std, 1.0)]
    starts = pu.starts_of(new, first)
    q = _bf16(rng, (int(starts[-1]) + behind, h, d), std)
    return cache, dense, starts, q


def _run(cache, dense, starts, q, scale=0.0, fill=np.nan, out=None):
    kp, vp = (dev(cache.pages_of(x, fill)) for x in dense)
    got = sd.paged_attention(dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens), scale, out)
    sd.sdpa_device_check()
    return got


def _check(got, cache, dense, starts, q, scale=0.0):
    ref, bound = pu.attention(q, *dense, starts, np.maximum(cache.lens, 0), scale)
    got = host(got)
    rows = ~np.isnan(ref)
    assert np.all(np.isfinite(got[rows]))
    excess = np.abs(got - ref)[rows] - bound[rows]
    assert excess.max(initial=-1.0) <= 0, (excess.max(), np.abs(got - ref)[rows].max())


SEQS = [([1], [1]), ([1], [63]), ([1], [64]), ([1], [65]), ([1], [300]), ([5], [5]), ([130], [130]), ([70], [400]),
        ([1, 1, 1], [1, 129, 1000]), ([3, 0, 40, 1, 0], [17, 90, 40, 700, 0]), ([4, 1, 6], [2, 0, 6])]


@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("new,lens", SEQS)
def test_attention_lengths(d, new, lens):
    """Single tokens, chunks and whole prompts; tiles and pages that end
    inside; empty sequences; more new tokens than positions."""
    rng = np.random.default_rng(100 + d + sum(new) + 7 * sum(lens))
    case = _case(rng, new, lens, 4, 2, d, 16)
    _check(_run(*case), *case)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 512])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
def test_attention_page_sizes(d, page):
    rng = np.random.default_rng(200 + d + page)
    case = _case(rng, [2, 33, 1], [page - 1, 3 * page + 5, 777], 4, 2, d, page)
    _check(_run(*case), *case)


@pytest.mark.parametrize("h,h_kv", [(1, 1), (8, 8), (16, 4), (6, 2), (5, 1), (14, 2), (33, 1), (128, 1), (256, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_head_groups(d, h, h_kv):
    """Groups that divide the 128 rows of a tile and groups that do not."""
    rng = np.random.default_rng(300 + d + h)
    case = _case(rng, [1, 7, 45], [200, 330, 45], h, h_kv, d, 32)
    _check(_run(*case), *case)


@pytest.mark.parametrize("d,h,h_kv,new,lens", [
    (128, 8, 1, [1], [20000]),                                   # one walk cut into many runs
    (64, 4, 4, [1, 1, 1, 1], [5000, 3, 9000, 64]),
    (128, 4, 1, [96, 1], [4000, 7000]),                          # rows of several tiles, each cut
    (256, 2, 1, [3], [12000]),
    (128, 32, 1, [1], [20000]),                                  # pieces that come in a few at a time
    (256, 16, 1, [2, 1], [9000, 5000]),
    (64, 33, 1, [1, 1], [9000, 4100]),                           # groups wider than a quarter tile
    (128, 16, 1, [1], [20000]),
    (256, 16, 1, [1, 1], [12000, 3000]),
    (16, 8, 2, [4], [30000]),
    (32, 3, 1, [200], [3000])])
def test_attention_split_walks(d, h, h_kv, new, lens):
    rng = np.random.default_rng(400 + d + h)
    case = _case(rng, new, lens, h, h_kv, d, 64)
    _check(_run(*case), *case)


def test_attention_uneven_walks_fill_every_run():
    """A prompt's walks from one key tile to many, among single tokens over
    long caches: units are cut by what they are expected to take."""
    rng = np.random.default_rng(512)
    new = [700] + [1] * 12 + [90]
    lens = [700] + [int(x) for x in rng.integers(1500, 6000, size=12)] + [2500]
    case = _case(rng, new, lens, 16, 4, 64, 64)
    _check(_run(*case), *case)


def test_attention_one_workspace_for_calls_of_all_shapes():
    """A workspace that holds other calls' leftovers, or anything."""
    import torch
    rng = np.random.default_rng(513)
    cases = [_case(rng, new, lens, h, h_kv, d, 32) for new, lens, h, h_kv, d in
             (([1], [4000], 8, 1, 128), ([40, 1], [300, 5000], 4, 2, 64), ([3], [9000], 2, 2, 256),
              ([130], [900], 6, 2, 32))]
    ready = []
    for cache, dense, starts, q in cases:
        kp, vp = (dev(cache.pages_of(x, np.nan)) for x in dense)
        args = (dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
        ready.append((args, sd.paged_attention(*args)))
    size = max(sd.paged_workspace(a[0], a[1], a[3]).numel() for a, _ in ready)
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            for args, want in ready:
                assert torch.equal(_raw(sd.paged_attention(*args, workspace=ws)), _raw(want))
    sd.sdpa_device_check()


@pytest.mark.parametrize("d,h,h_kv,new,lens", [
    (64, 2, 2, [69], [26595]),              # 52 pieces of 69 rows
    (128, 16, 4, [32], [8192]),             # 8 of 128 rows, 4 times
    (16, 128, 1, [1], [6000]),              # 24 of 128 rows
    (32, 3, 1, [33], [12000]),              # 24 of 99 rows
    (256, 5, 1, [3], [30000]),              # 59 of 15 rows
    (64, 16, 1, [1, 1], [33000, 20000]),    # 129 and 79 of 16 rows
    (128, 1, 1, [1], [40000]),              # 157 of a single row: slices of columns
    (16, 32, 16, [1, 1], [30000, 100]),     # more than there are runs: cut by weight
    (64, 16, 4, [1, 1], [70000, 300]),
    (256, 16, 2, [17], [20000]),
])
def test_attention_in_slices(d, h, h_kv, new, lens):
    """Units of so many pieces that several runs merge them, in a workspace that
    holds anything; the same bits again, called and replayed."""
    import torch
    rng = np.random.default_rng(520 + d + sum(lens))
    case = _case(rng, new, lens, h, h_kv, d, 64)
    cache, dense, starts, q = case
    kp, vp = (dev(cache.pages_of(x, np.nan)) for x in dense)
    args = (dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    ws = sd.paged_workspace(args[0], kp, args[3])
    ws.fill_(0xff)
    out = torch.empty_like(args[0])
    sd.paged_attention(*args, out=out, workspace=ws)
    sd.sdpa_device_check()
    _check(out, *case)
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            sd.paged_attention(*args, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(_raw(out), _raw(want))
    sd.sdpa_device_check()


def test_attention_many_sequences():
    """More sequences than threads in a block, most of them short, some empty."""
    rng = np.random.default_rng(500)
    new = rng.integers(0, 3, size=700)
    lens = rng.integers(0, 60, size=700)
    lens[::97] = 900
    case = _case(rng, new, lens, 4, 2, 64, 16)
    _check(_run(*case), *case)


def test_attention_whole_prompt_over_many_tiles():
    rng = np.random.default_rng(501)
    case = _case(rng, [1000, 37], [1000, 1500], 6, 3, 128, 64)
    _check(_run(*case), *case)


@pytest.mark.parametrize("fill", [np.nan, np.inf, -np.inf, 3e38])
def test_attention_ignores_rows_past_the_length(fill):
    rng = np.random.default_rng(502)
    for d in (32, 64, 128, 256):
        case = _case(rng, [1, 9, 2], [70, 9, 129], 4, 2, d, 32)
        got = _run(*case, fill=fill)
        _check(got, *case)


def test_attention_sharp_and_unscaled():
    """Scores that grow along the walk (the running maximum moves from tile to
    tile) and a scale of the caller's."""
    rng = np.random.default_rng(503)
    cache, (k, v), starts, q = _case(rng, [1, 20], [3000, 500], 4, 2, 64, 64, std=0.5)
    k = [synthetic.round_to_bf16((x * np.linspace(0.2, 3.0, len(x))[:, None, None]).astype(np.float32)) for x in k]
    case = (cache, [k, v], starts, q)
    for scale in (0.5, 1.0):
        _check(_run(*case, scale=scale), *case, scale=scale)


def test_attention_leaves_other_rows_alone():
    """Rows before the first and behind the last sequence are not written;
    rows at negative positions are zero."""
    rng = np.random.default_rng(504)
    case = _case(rng, [3, 5], [40, 2], 4, 2, 64, 16, first=2, behind=4)
    out = dev(np.full(case[3].shape, 7.0, np.float32))
    got = host(_run(*case, out=out))
    assert np.all(got[:2] == 7.0) and np.all(got[10:] == 7.0)
    assert np.all(got[5:8] == 0.0)
    _check(out, *case)


def test_attention_takes_strided_queries():
    rng = np.random.default_rng(505)
    cache, dense, starts, q = _case(rng, [1, 30], [90, 300], 8, 2, 64, 16)
    wide = dev(_bf16(rng, (q.shape[0], 12, 64)))
    wide[:, :8] = dev(q)
    kp, vp = (dev(cache.pages_of(x, np.nan)) for x in dense)
    rest = (kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    a, b = sd.paged_attention(wide[:, :8], *rest), sd.paged_attention(dev(q), *rest)
    sd.sdpa_device_check()
    assert np.array_equal(host(a), host(b))


def test_attention_shared_pages():
    """Two sequences whose tables name the same pages for a common prefix."""
    rng = np.random.default_rng(506)
    cache, (k, v), starts, q = _case(rng, [2, 1], [100, 100], 4, 2, 64, 16)
    cache.table[1, :4] = cache.table[0, :4]
    k[1][:64], v[1][:64] = k[0][:64], v[0][:64]
    case = (cache, [k, v], starts, q)
    _check(_run(*case), *case)


def test_attention_repeats_bit_for_bit():
    import torch
    rng = np.random.default_rng(507)
    cache, dense, starts, q = _case(rng, [1, 60, 1], [6000, 900, 3000], 8, 2, 128, 64)
    kp, vp = (dev(cache.pages_of(x, np.nan)) for x in dense)
    args = (dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    first = sd.paged_attention(*args)
    ws = sd.paged_workspace(args[0], kp, args[3])
    for _ in range(5):
        assert torch.equal(_raw(sd.paged_attention(*args, workspace=ws)), _raw(first))
    sd.sdpa_device_check()


def test_attention_bad_page_is_reported_and_reads_as_zeros():
    rng = np.random.default_rng(508)
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        cache, (k, v), starts, q = _case(rng, [1, 1], [100, 100], 4, 2, 64, 16)
        kp, vp = (dev(cache.pages_of(x, np.nan)) for x in (k, v))
        cache.table[1, 2] = bad
        got = sd.paged_attention(dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
        with pytest.raises(sd.SdpaError) as e:
            sd.sdpa_device_check()
        assert e.value.status == 7
        sd.sdpa_device_check()                                   # cleared
        k[1][32:48], v[1][32:48] = 0, 0
        _check(got, cache, [k, v], starts, q)


def test_attention_clamps_what_the_arrays_say():
    """Lengths past the table and negative ones, row offsets past the rows:
    everything stays inside the buffers."""
    rng = np.random.default_rng(509)
    cache, (k, v), starts, q = _case(rng, [2, 2, 2], [64, 30, 64], 4, 2, 64, 16)
    cap = cache.per_seq * 16
    kp, vp = (dev(cache.pages_of(x, 0.0)) for x in (k, v))
    cache.table[0, :] = cache.table[0, 0]
    lens = np.array([10 ** 9, -5, 64], np.int32)
    out = dev(np.full(q.shape, 7.0, np.float32))
    sd.paged_attention(dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(lens), out=out)
    sd.sdpa_device_check()
    got = host(out)
    assert np.all(got[2:4] == 0.0)
    dense = [[np.tile(x[0][:16], (cap // 16, 1, 1)), x[1][:0], x[2]] for x in (k, v)]
    cache.lens = np.array([cap, 0, 64], np.int32)
    _check(out, cache, dense, starts, q)
    # offsets outside the rows: the rows that exist are the sequence's last ones
    sd.paged_attention(dev(q), kp, vp, dev_int(cache.table), dev_int(np.array([-9, -3, 4, 90], np.int32)),
                       dev_int(np.array([64, 30, 64], np.int32)))
    sd.sdpa_device_check()


def test_attention_far_pages():
    """Pages whose element offsets pass 32 bits."""
    import torch
    h_kv, page, d = 8, 256, 128
    n_pages = (1 << 32) // (h_kv * page * d) + 3
    rng = np.random.default_rng(510)
    kp = torch.empty((n_pages, h_kv, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = np.array([[n_pages - 1, 0], [n_pages - 2, n_pages // 2 + 1]], np.int32)
    lens, new = np.array([300, 400], np.int32), [2, 1]
    starts = pu.starts_of(new)
    k, v = ([_bf16(rng, (n, h_kv, d)) for n in lens] for _ in range(2))
    f = pu.freqs_of(d)
    # through the append: every position written, then read
    all_new = pu.starts_of(lens)
    rows_k, rows_v = dev(np.concatenate(k)), dev(np.concatenate(v))
    tab, ln = dev_int(table), dev_int(lens)
    assert sd.paged_append(None, rows_k, rows_v, kp, vp, tab, dev_int(all_new), ln) is None
    q = _bf16(rng, (3, h_kv, d))
    got = sd.paged_attention(dev(q), kp, vp, tab, dev_int(starts), ln)
    sd.sdpa_device_check()
    ref, bound = pu.attention(q, k, v, starts, lens)
    assert np.all(np.abs(host(got) - ref) <= bound)
    assert len(f) == d // 2


def test_attention_no_tokens():
    rng = np.random.default_rng(511)
    cache, dense, starts, q = _case(rng, [0, 0], [40, 0], 4, 2, 64, 16, behind=3)
    out = dev(np.full(q.shape, 7.0, np.float32))
    assert np.all(host(_run(cache, dense, starts, q, out=out)) == 7.0)
    empty = _run(cache, dense, starts, q[:0])
    assert empty.shape == (0, 4, 64)
    kp, vp = (dev(cache.pages_of(x, 0.0)) for x in dense)
    rest = (kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    assert sd.paged_append(empty, empty[:, :2], empty[:, :2], *rest).shape == (0, 4, 64)
    sd.sdpa_device_check()


# --------------------------------------------------------------------- append
def _append_case(rng, new, lens, h, h_kv, d, page, first=0, behind=0):
    cache = pu.Cache(rng, lens, h_kv, d, page)
    starts = pu.starts_of(new, first)
    t = int(starts[-1]) + behind
    return cache, starts, _bf16(rng, (t, h, d)), _bf16(rng, (t, h_kv, d)), _bf16(rng, (t, h_kv, d))


def _check_append(cache, starts, q, k, v, freqs, interleaved, before, after, q_out, q_before):
    """before, after: (k_pages, v_pages) as arrays; q_before: q_out's rows of
    no sequence."""
    lens = np.clip(cache.lens, 0, cache.per_seq * cache.page)
    where = pu.positions_of(len(q), starts, lens)
    rows = [i for i, p in enumerate(where) if p is not None]
    pos = np.array([where[i] for i in rows])
    want, bound = pu.rotate(q[rows], pos, freqs, interleaved)
    assert np.all(np.abs(q_out[rows] - want) <= bound)
    other = [i for i, p in enumerate(where) if p is None]
    assert np.array_equal(q_out[other], q_before[other])
    kw, kb = pu.rotate(k[rows], pos, freqs, interleaved)
    seq_of = {i: s for s in range(len(lens)) for i in range(starts[s], starts[s + 1])}
    kept = np.ones(before[0].shape[:1] + before[0].shape[2:3], bool)
    for x, i in enumerate(rows):
        if pos[x] < 0:
            continue
        page, slot = cache.table[seq_of[i], pos[x] // cache.page], pos[x] % cache.page
        assert np.all(np.abs(after[0][page, :, slot] - kw[x]) <= kb[x])
        assert np.array_equal(after[1][page, :, slot], v[i])
        kept[page, slot] = False
    for a, b in zip(before, after):
        assert np.array_equal(a.transpose(0, 2, 1, 3)[kept], b.transpose(0, 2, 1, 3)[kept])


def _run_append(rng, case, d_rot, interleaved, in_place=False):
    cache, starts, q, k, v = case
    f = pu.freqs_of(d_rot)
    shape = (cache.n_pages, cache.h_kv, cache.page, cache.d)
    before = [_bf16(rng, shape) for _ in range(2)]
    kp, vp = dev(before[0]), dev(before[1])
    qd = dev(q)
    q_out = qd if in_place else dev(np.full(q.shape, 7.0, np.float32))
    q_before = host(q_out)
    sd.paged_append(qd, dev(k), dev(v), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens),
                    dev(f, "f32") if d_rot else None, interleaved, q_out)
    sd.sdpa_device_check()
    _check_append(cache, starts, q, k, v, f, interleaved, before, (host(kp), host(vp)), host(q_out), q_before)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,d_rot", [(16, 16), (32, 16), (64, 64), (64, 0), (128, 128), (128, 48), (256, 256)])
def test_append_head_sizes(d, d_rot, interleaved):
    rng = np.random.default_rng(600 + d + d_rot)
    case = _append_case(rng, [1, 17, 0, 3], [5, 17, 40, 900], 6, 2, d, 16)
    _run_append(rng, case, d_rot, interleaved)


@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("h,h_kv", [(1, 1), (5, 1), (16, 16), (128, 1)])
def test_append_head_counts_and_pages(h, h_kv, page):
    rng = np.random.default_rng(700 + h + page)
    _run_append(rng, _append_case(rng, [9, 1, 2], [300, 1, 77], h, h_kv, 64, page), 64, False)


def test_append_edges():
    """Rows of no sequence, more new tokens than positions, an empty
    sequence, in place."""
    rng = np.random.default_rng(701)
    case = _append_case(rng, [4, 0, 6, 1], [2, 9, 30, 64], 4, 2, 64, 16, first=3, behind=5)
    _run_append(rng, case, 64, False)
    _run_append(rng, case, 32, True, in_place=True)


def test_append_many_tokens_and_sequences():
    rng = np.random.default_rng(702)
    new = rng.integers(0, 5, size=900)
    lens = new + rng.integers(0, 30, size=900)
    _run_append(rng, _append_case(rng, new, lens, 2, 1, 32, 8), 32, False)
    _run_append(rng, _append_case(rng, [1500, 1], [1500, 2000], 2, 2, 64, 64), 64, True)


@pytest.mark.parametrize("start", [0, 4095, 4096, 131071, (1 << 24) + 1, (1 << 29) - 9])
def test_append_far_positions(start):
    """Angles of positions that fp32 products alone would lose.  One page is
    handed out again and again: only the last page's worth of tokens counts."""
    import torch
    rng = np.random.default_rng(703)
    d, page, n = 64, 1 << 20, 8
    length = start + n
    per_seq = length // page + 1
    table = np.zeros((1, per_seq), np.int32)
    q, k, v = (_bf16(rng, (n, 1, d)) for _ in range(3))
    kp = torch.zeros((1, 1, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    f = pu.freqs_of(d)
    q_out = sd.paged_append(dev(q), dev(k), dev(v), kp, vp, dev_int(table), dev_int(np.array([0, n], np.int32)),
                            dev_int(np.array([length], np.int32)), dev(f, "f32"))
    sd.sdpa_device_check()
    pos = np.arange(start, start + n)
    for got, x in ((host(q_out), q), (host(kp[0, 0, pos % page][:, None]), k)):
        want, bound = pu.rotate(x, pos, f, False)
        assert np.all(np.abs(got - want) <= bound)


def test_append_bad_page_is_reported_and_skipped():
    import torch
    rng = np.random.default_rng(704)
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        cache, starts, q, k, v = _append_case(rng, [1, 1], [20, 20], 4, 2, 64, 16)
        cache.table[1, 1] = bad
        kp = torch.full((cache.n_pages, 2, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        vp = kp.clone()
        q_out = sd.paged_append(dev(q), dev(k), dev(v), kp, vp, dev_int(cache.table), dev_int(starts),
                                dev_int(cache.lens), dev(pu.freqs_of(64), "f32"))
        with pytest.raises(sd.SdpaError) as e:
            sd.sdpa_device_check()
        assert e.value.status == 7
        want, bound = pu.rotate(q, np.array([19, 19]), pu.freqs_of(64), False)
        assert np.all(np.abs(host(q_out) - want) <= bound)
        changed = (host(kp) != 7.0).any(axis=(1, 3))
        assert changed.sum() == 1 and changed[cache.table[0, 1], 3]


# ------------------------------------------------------------ the two together
def _weights(rng, dm, h, h_kv, d):
    return (_bf16(rng, (dm, (h + 2 * h_kv) * d), dm ** -0.5), _bf16(rng, (h * d, dm), (h * d) ** -0.5))


class _Layer:
    """One attention layer as a serving loop runs it: projection, append,
    attention, output projection, on buffers it keeps."""

    def __init__(self, rng, cache, h, h_kv, d, dm, t):
        import torch
        self.h, self.h_kv, self.d, self.dm = h, h_kv, d, dm
        self.w, self.wo = (dev(x) for x in _weights(rng, dm, h, h_kv, d))
        shape = (cache.n_pages, h_kv, cache.page, d)
        self.kp = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        self.table = dev_int(cache.table)
        self.freqs = dev(pu.freqs_of(d), "f32")
        self.qkv = torch.empty((t, (h + 2 * h_kv) * d), dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda")
        self.out, self.y = torch.empty_like(self.q), torch.empty((t, dm), dtype=torch.bfloat16, device="cuda")
        self.ws = sd.paged_workspace(self.q, self.kp, self.table)

    def step(self, x, starts, lens, stream=None):
        t, h, h_kv, d = x.shape[0], self.h, self.h_kv, self.d
        sd.linear_forward(x, self.w, self.qkv, t, self.qkv.shape[1], self.dm, stream)
        rows = self.qkv.view(-1, h + 2 * h_kv, d)[:t]
        sd.paged_append(rows[:, :h], rows[:, h:h + h_kv], rows[:, h + h_kv:], self.kp, self.vp, self.table, starts,
                        lens, self.freqs, q_out=self.q[:t], stream=stream)
        sd.paged_attention(self.q[:t], self.kp, self.vp, self.table, starts, lens, out=self.out[:t],
                           workspace=self.ws, stream=stream)
        sd.linear_forward(self.out, self.wo, self.y, t, self.dm, h * d, stream)
        return self.y[:t]


def _serve(rng, lens, schedule, h=8, h_kv=2, d=64, dm=256, page=16):
    """Feeds the sequences' inputs in the given chunks.  Returns, over the
    packed whole sequences, the rotated queries and the attention's rows, and
    each sequence's cached keys and values."""
    cache = pu.Cache(rng, lens, h_kv, d, page)
    layer = _Layer(rng, cache, h, h_kv, d, dm, sum(lens))
    xs = [_bf16(rng, (n, dm)) for n in lens]
    done = [0] * len(lens)
    q, out = [[] for _ in lens], [[] for _ in lens]
    for chunk in schedule:
        new = [min(c, n - a) for c, n, a in zip(chunk, lens, done)]
        x = np.concatenate([xs[s][done[s]:done[s] + n] for s, n in enumerate(new)])
        done = [a + n for a, n in zip(done, new)]
        starts = pu.starts_of(new)
        layer.step(dev(x), dev_int(starts), dev_int(np.array(done, np.int32)))
        for part, rows in ((q, host(layer.q)), (out, host(layer.out))):
            for s in range(len(lens)):
                part[s].append(rows[starts[s]:starts[s + 1]])
    sd.sdpa_device_check()
    assert done == list(lens)

    def cached(pages):
        rows = [[pages[cache.table[s, j // page], :, j % page] for j in range(n)] for s, n in enumerate(lens)]
        return [np.array(r) for r in rows]

    flat = [np.concatenate([np.concatenate(x) for x in part]) for part in (q, out)]
    return flat[0], flat[1], cached(host(layer.kp)), cached(host(layer.vp)), layer


@pytest.mark.parametrize("schedule", [[[90, 33, 1]], [[40, 1, 0], [7, 30, 1], [43, 2, 0]],
                                      [[80, 20, 0]] + [[1, 1, 1]] * 13], ids=["whole", "chunks", "tokens"])
def test_serving_in_chunks(schedule):
    """Prompts fed whole, in odd chunks and token by token through projection,
    append, attention and output projection: every step's attention is that of
    the whole sequence's causal rows over what the cache holds at the end, and
    the cached keys are the rotated columns of the projection."""
    lens = [90, 33, 1]
    q, out, k, v, layer = _serve(np.random.default_rng(800), lens, schedule)
    ref, bound = pu.attention(q, k, v, pu.starts_of(lens), lens)
    assert np.all(np.abs(out - ref) <= bound)
    # the projection of the same inputs, with its own bf16 rounding taken from the GPU
    rng = np.random.default_rng(800)
    cache = pu.Cache(rng, lens, 2, 64, 16)
    _weights(rng, 256, 8, 2, 64)
    x = np.concatenate([_bf16(rng, (n, 256)) for n in lens])
    import torch
    rows = torch.empty((sum(lens), 12 * 64), dtype=torch.bfloat16, device="cuda")
    sd.linear_forward(dev(x), layer.w, rows, sum(lens), 12 * 64, 256)
    rows = host(rows).reshape(-1, 12, 64)
    pos = np.concatenate([np.arange(n) for n in lens])
    want, slack = pu.rotate(rows[:, :10], pos, pu.freqs_of(64), False)
    assert cache.n_pages > 0
    # a projected row is the same whatever rows come with it, to its rounding
    slack = slack + 2 * 2.0 ** -7 * (np.abs(want) + np.abs(rows[:, :10]).max(axis=-1, keepdims=True))
    assert np.all(np.abs(np.concatenate([q, np.concatenate(k)], axis=1) - want) <= slack)


def test_paged_equals_dense_attention():
    """Without rotation, one kv head a query head: the causal forward and the
    decoding step over dense tensors."""
    rng = np.random.default_rng(801)
    b, h, n, d = 2, 4, 200, 64
    q, k, v = (_bf16(rng, (b, h, n, d)) for _ in range(3))
    dense = host(sd.attention(dev(q), dev(k), dev(v), sd.SDPA_MASK_CAUSAL))
    cache = pu.Cache(rng, [n] * b, h, d, 32)
    rows = [dev(x.transpose(0, 2, 1, 3).reshape(b * n, h, d)) for x in (q, k, v)]
    kp, vp = (dev(np.full((cache.n_pages, h, 32, d), np.nan, np.float32)) for _ in range(2))
    table, starts, lens = dev_int(cache.table), dev_int(pu.starts_of([n] * b)), dev_int(cache.lens)
    rq = sd.paged_append(*rows, kp, vp, table, starts, lens)
    assert np.array_equal(host(rq), host(rows[0]))
    got = host(sd.paged_attention(rq, kp, vp, table, starts, lens)).reshape(b, n, h, d).transpose(0, 2, 1, 3)
    sd.sdpa_device_check()
    ref, bound = pu.attention(host(rq), *([list(x.transpose(0, 2, 1, 3)) for x in (k, v)]), pu.starts_of([n] * b),
                              cache.lens)
    bound = bound.reshape(b, n, h, d).transpose(0, 2, 1, 3)
    assert np.all(np.abs(got - dense) <= 2 * bound)              # each is within its bound of the exact value
    step = host(sd.decode_step(dev(q[:, :, -3:]), dev(k), dev(v)))
    assert np.all(np.abs(got[:, :, -3:] - step) <= 2 * bound[:, :, -3:])


def test_captured_step_follows_the_lengths():
    """One captured step (projection, append, attention, projection) replayed
    while the lengths grow equals eager steps, bit for bit."""
    import torch
    lens = [70, 300]

    def build():
        rng = np.random.default_rng(802)
        cache = pu.Cache(rng, [n + 8 for n in lens], 2, 64, 16)
        layer = _Layer(rng, cache, 8, 2, 64, 256, sum(lens))
        layer.step(dev(_bf16(rng, (sum(lens), 256))), dev_int(pu.starts_of(lens)), dev_int(np.array(lens, np.int32)))
        return layer, [dev(_bf16(rng, (2, 256))) for _ in range(4)]

    eager, xs = build()
    starts = dev_int(np.array([0, 1, 2], np.int32))
    want = [eager.step(x, starts, dev_int(np.array(lens, np.int32) + i + 1)).clone() for i, x in enumerate(xs)]
    graphed, xs = build()
    x, ln = xs[0].clone(), dev_int(np.array(lens, np.int32) + 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphed.step(x, starts, ln)                               # warm-up; position len is written again below
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        graphed.step(x, starts, ln)
    for i, row in enumerate(xs):
        x.copy_(row)
        ln.copy_(dev_int(np.array(lens, np.int32) + i + 1))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(_raw(graphed.y[:2]), _raw(want[i])), i
    sd.sdpa_device_check()


def test_two_streams_with_a_workspace_each():
    import torch
    rng = np.random.default_rng(803)
    sides = []
    for n in (5000, 3000):
        cache, dense, starts, q = _case(rng, [2, 1], [n, 100], 8, 2, 128, 64)
        kp, vp = (dev(cache.pages_of(x, np.nan)) for x in dense)
        args = (dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
        sides.append((args, sd.paged_attention(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (args, _, stream) in enumerate(sides):
            outs[i].append(sd.paged_attention(*args, stream=stream))
    torch.cuda.synchronize()
    sd.sdpa_device_check()
    for i, (_, want, _) in enumerate(sides):
        for o in outs[i]:
            assert torch.equal(_raw(o), _raw(want))


def test_slices_beside_other_work():
    """Units merged by several runs on two streams at once, while matrix products
    on a third hold SMs: runs wait for runs that may not have begun."""
    import torch
    rng = np.random.default_rng(804)
    jobs = []
    for new, lens, h, h_kv, d in (([69], [26595], 2, 2, 64), ([1, 1], [70000, 300], 16, 4, 64)):
        cache = pu.Cache(rng, lens, h_kv, d, 64)
        dense = [[_bf16(rng, (n, h_kv, d)) for n in lens] for _ in range(2)]
        kp, vp = (dev(cache.pages_of(x, 0.0)) for x in dense)
        q = dev(_bf16(rng, (sum(new), h, d)))
        args = (q, kp, vp, dev_int(cache.table), dev_int(pu.starts_of(new)), dev_int(cache.lens))
        want = sd.paged_attention(*args)
        jobs.append((args, want, sd.paged_workspace(q, kp, args[3]), torch.cuda.Stream(), []))
    a = torch.randn(4096, 4096, dtype=torch.bfloat16, device="cuda")
    c = torch.empty_like(a)
    third = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(60):
        with torch.cuda.stream(third):
            torch.mm(a, a, out=c)
        for args, _, ws, stream, outs in jobs:
            outs.append(sd.paged_attention(*args, workspace=ws, stream=stream))
    torch.cuda.synchronize()
    sd.sdpa_device_check()
    for _, want, _, _, outs in jobs:
        for out in outs:
            assert torch.equal(_raw(out), _raw(want))


def test_inputs_written_just_before_the_call():
    """Lengths, tables and queries written by kernels of the same stream right
    before each call."""
    import torch
    rng = np.random.default_rng(804)
    cache, dense, starts, q = _case(rng, [1, 40], [700, 300], 4, 2, 64, 16)
    kp, vp = (dev(cache.pages_of(x, 0.0)) for x in dense)
    qd, table, st = dev(q), dev_int(cache.table), dev_int(starts)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    qw, tw = torch.empty_like(qd), torch.empty_like(table)
    for r, now in enumerate(([700, 300], [64, 40], [333, 299])):
        sign = 1.0 if r % 2 == 0 else -1.0
        for i, n in enumerate(now):
            lens[i:i + 1].fill_(n)
        tw.copy_(table)
        torch.mul(qd, sign, out=qw)
        got = sd.paged_attention(qw, kp, vp, tw, st, lens)
        cut = [[x[s][:now[s]] for s in range(2)] for x in dense]
        ref, bound = pu.attention(q * np.float32(sign), *cut, starts, now)
        assert np.all(np.abs(host(got) - ref) <= bound), r
        lens.zero_()
        tw.fill_(-1)
    sd.sdpa_device_check()


def test_helpers_refuse_other_types_and_layouts():
    import torch
    rng = np.random.default_rng(805)
    cache, dense, starts, q = _case(rng, [1], [40], 4, 2, 64, 16)
    kp, vp = (dev(cache.pages_of(x, 0.0)) for x in dense)
    good = [dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens)]
    sd.paged_attention(*good)

    def refused(i, x, call=sd.paged_attention, args=good):
        bad = list(args)
        bad[i] = x
        with pytest.raises(sd.SdpaError) as e:
            call(*bad)
        assert e.value.status == 1

    refused(0, good[0].half())
    refused(0, good[0].float())
    refused(0, good[0][..., ::2])
    refused(0, good[0].cpu())
    refused(0, good[0][..., :32].contiguous())
    refused(1, kp.transpose(1, 2))
    refused(2, vp[:, :1].contiguous())
    refused(3, good[3].long())
    refused(4, good[4].long())
    refused(4, good[4][:1])
    refused(5, good[5].cpu())
    kv = dev(_bf16(rng, (1, 2, 64)))
    good2 = [good[0], kv, kv] + good[1:]
    sd.paged_append(*good2)
    refused(1, kv[:, :1], sd.paged_append, good2)
    refused(2, kv.float(), sd.paged_append, good2)
    with pytest.raises(sd.SdpaError):
        sd.paged_append(*good2, rope_freqs=torch.zeros(32, dtype=torch.float64, device="cuda"))
    with pytest.raises(sd.SdpaError):
        sd.paged_attention(*good, out=torch.empty((1, 4, 64), dtype=torch.float32, device="cuda"))
    torch.cuda.synchronize()
