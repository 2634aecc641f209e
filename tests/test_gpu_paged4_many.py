"""Attention over the cache in 4 bits for sequences of many rows (chunks of a prompt
and whole prompts, alone and among single tokens), and what the two kernels of such a
call share: the workspace, captured graphs, streams, bad pages.  Against the plain
fp64 implementation and bounds of paged4_util.py."""
import ctypes
import os
import subprocess
import tempfile
import time

import numpy as np
import pytest

import paged4_util as p4
import paged_util as pu
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int, host
from test_gpu_paged4 import HEADS, _args, _bf16, _bytes, _case, _check, _kw, _read, _run
from transformer_scaled_dot_02_gb300 import build as sd_build

pytestmark = pytest.mark.gpu


# Row tiles of 128 and 256 rows that are full, begun and missed by one; walks that are
# cut and that are not; rows at negative positions, whole tiles of them, no key at all.
MANY = [([128], [128]), ([64], [64]), ([129, 1], [4000, 1]), ([127, 0, 65], [500, 70, 65]), ([257, 1, 300], [257, 900, 2000]),
        ([600], [600]), ([600], [100]), ([400, 9], [0, 40]), ([33] * 9, [33, 34, 100, 200, 300, 0, 20, 63, 64])]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("new,lens", MANY)
def test_lengths(d, new, lens):
    rng = np.random.default_rng(4000 + d + sum(new) + 7 * sum(lens))
    c = _case(rng, new, lens, 4, 2, d, 16, first=3, behind=2)
    _check(_run(c), c)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (16, 32), (256, 128), (32, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (128, 0), (129, 127), (500, 64), (200, 300), (5000, 7), (40, 100000)])
def test_windows(d, page, window, sinks):
    rng = np.random.default_rng(4100 + d + window + sinks)
    c = _case(rng, [300, 1, 70, 150], [1300, 700, 300, 100], 6, 2, d, page, window=window, sinks=sinks)
    _check(_run(c), c)


@pytest.mark.parametrize("h,h_kv", [(5, 1), (33, 1), (128, 1), (24, 8), (1, 1), (3, 3)])
@pytest.mark.parametrize("d", [128, 256])
def test_head_groups(d, h, h_kv):
    """Tiles that end inside a token's group of heads."""
    rng = np.random.default_rng(4200 + d + h)
    c = _case(rng, [100, 3, 37], [300, 500, 37], h, h_kv, d, 32)
    _check(_run(c), c)


@pytest.mark.parametrize("d,h,h_kv,new,lens", [
    (128, 4, 1, [200], [12000]), (64, 2, 1, [130, 1], [30000, 9000]), (256, 2, 1, [90], [9000]),
    (32, 8, 1, [40], [20000]), (16, 3, 1, [300], [8000])])
def test_walks_in_many_pieces(d, h, h_kv, new, lens):
    rng = np.random.default_rng(4300 + d)
    c = _case(rng, new, lens, h, h_kv, d, 64)
    _check(_run(c), c)


def test_one_sequence_of_many_rows_in_few_tokens():
    """No more tokens than sequences, all of them of one: the few-rows kernel's."""
    rng = np.random.default_rng(4400)
    c = _case(rng, [0] * 20 + [30] + [0] * 19, [5] * 20 + [700] + [9] * 19, 8, 2, 64, 16)
    _check(_run(c), c)


def test_many_sequences():
    rng = np.random.default_rng(4401)
    lens = [int(x) for x in rng.integers(0, 300, size=500)]
    new = [int(x) for x in rng.integers(0, 7, size=500)]
    c = _case(rng, new, lens, 8, 1, 32, 16)
    _check(_run(c), c)


def test_rows_that_are_not_finite_stay_their_own():
    rng = np.random.default_rng(4402)
    c = _case(rng, [140], [600], 4, 2, 128, 32)
    want = host(_run(c))
    q = c["q"].copy()
    q[77, 1], q[3, 3, 5] = np.nan, np.inf
    got = host(_run(dict(c, q=q)))
    other = np.ones(got.shape[:2], bool)
    other[77, 1] = other[3, 3] = False
    assert np.array_equal(got[other], want[other]) and np.isnan(got[77, 1]).all()


def test_wide_range_of_queries_and_a_scale():
    rng = np.random.default_rng(4403)
    c = _case(rng, [200], [900], 4, 2, 64, 16)
    c["q"][:, 0] *= np.float32(2.0 ** 40)
    c["q"][:, 2] *= np.float32(2.0 ** -60)
    c["q"][5] = 0.0
    _check(_run(c, scale=2.0 ** -41), c, scale=2.0 ** -41)


def test_repeats_bit_by_bit():
    """The same call again and again, in workspaces that hold anything."""
    import torch
    rng = np.random.default_rng(4500)
    cases = [_case(rng, new, lens, h, h_kv, d, 32) for new, lens, h, h_kv, d in
             (([300, 1, 1], [9000, 4000, 60], 8, 2, 128), ([500], [500], 16, 2, 64), ([100, 90], [5000, 90], 2, 1, 256))]
    ready = [(_args(c), _kw(c)) for c in cases]
    want = [sd.paged4_attention(*a, **kw) for a, kw in ready]
    for c, w in zip(cases, want):
        _check(w, c)
    size = max(sd.paged4_workspace(a[0], a[1], a[3]).numel() for a, _ in ready)
    for fill in (0x00, 0xff, 0x41):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(10):
            for (args, kw), w in zip(ready, want):
                assert torch.equal(sd.paged4_attention(*args, **kw, workspace=ws), w)
    sd.sdpa_device_check()


def test_repeats_whichever_run_comes_last():
    """Units in two pieces, merged by the run of the one or of the other: copies of
    odd sizes in another stream change which of them is the last."""
    import torch
    rng = np.random.default_rng(4506)
    other, junk = torch.cuda.Stream(), torch.empty(2, 1 << 22, device="cuda")
    for new, lens, h, h_kv, d, window in (([700, 300], [1500, 4000], 12, 2, 128, 500), ([500], [500], 16, 2, 64, 0),
                                          ([2000], [2000], 4, 2, 32, 0)):
        c = _case(rng, new, lens, h, h_kv, d, 32, window=window, sinks=4 if window else 0)
        args, kw = _args(c), _kw(c)
        ws = sd.paged4_workspace(args[0], args[1], args[3])
        want = sd.paged4_attention(*args, **kw, workspace=ws)
        outs = [torch.empty_like(want) for _ in range(50)]
        for i in range(100):
            if i % 3 == 0:
                n = int(rng.integers(1 << 10, 1 << 22))
                with torch.cuda.stream(other):
                    junk[0, :n].copy_(junk[1, :n])
            sd.paged4_attention(*args, **kw, out=outs[i % 50], workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in outs)
    sd.sdpa_device_check()


def test_graphs_that_share_a_workspace_follow_starts_and_lengths():
    """Two graphs of calls of 200 rows, whose starts change between replays from one
    sequence's chunk to single tokens and back."""
    import torch
    rng = np.random.default_rng(4501)
    lens = [5000, 300, 900, 2000]
    c = _case(rng, [197, 1, 1, 1], lens, 8, 2, 64, 64)
    args = _args(c)
    ws = sd.paged4_workspace(args[0], args[1], args[3])
    outs = [torch.zeros(200, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.paged4_attention(*args, **_kw(c), out=outs[0], workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sd.paged4_attention(*args, **_kw(c), out=out, workspace=ws)
        graphs.append(g)
    for new, now in (([197, 1, 1, 1], lens), ([1, 1, 1, 1], lens), ([50, 60, 3, 87], [4000, 60, 900, 100]),
                     ([0, 0, 0, 0], lens), ([0, 200, 0, 0], [1, 299, 5, 7]), ([2, 2, 2, 2], [5000, 2, 1, 1999])):
        starts = pu.starts_of(new)
        args[4].copy_(dev_int(starts))
        args[5].copy_(dev_int(now))
        c["cache"].lens = np.asarray(now, np.int32)
        for g, out in zip(graphs, outs):
            out.fill_(7.0)
            for _ in range(2):
                g.replay()
        held = [[x[:n] for x, n in zip(h, now)] for h in c["held"]]
        for out in outs:
            _check(out, dict(c, held=held, starts=starts))
            assert bool((out[int(starts[-1]):] == 7.0).all())
    sd.sdpa_device_check()


def test_two_streams_at_once():
    import torch
    rng = np.random.default_rng(4502)
    cases = [_case(rng, [150, 1], [3000, 800], 8, 2, d, 32) for d in (16, 128)]
    ready = [(_args(c), _kw(c)) for c in cases]
    want = [sd.paged4_attention(*a, **kw) for a, kw in ready]
    spaces = [sd.paged4_workspace(a[0], a[1], a[3]) for a, _ in ready]
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    streams = [torch.cuda.Stream() for _ in ready]
    torch.cuda.synchronize()
    for i in range(8):
        for (a, kw), ws, out, stream in zip(ready, spaces, outs, streams):
            sd.paged4_attention(*a, **kw, out=out[i], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        assert all(torch.equal(x, w) for x in out)
    sd.sdpa_device_check()


def test_among_the_other_kernels():
    """Between launches that hold tensor memory too, in one stream and captured."""
    import torch
    rng = np.random.default_rng(4503)
    c = _case(rng, [300], [3000], 4, 2, 16, 16)
    args, kw = _args(c), _kw(c)
    want = sd.paged4_attention(*args, **kw)
    ws = sd.paged4_workspace(args[0], args[1], args[3])
    q = torch.randn(2, 4, 512, 64, device="cuda").bfloat16()
    got, outs = torch.empty_like(want), [torch.empty_like(q) for _ in range(2)]
    other = torch.empty_like(q)
    sd.sdpa_forward(q, q, q, other, 2, 4, 512, 512, 64, 64)

    def run():
        sd.sdpa_forward(q, q, q, outs[0], 2, 4, 512, 512, 64, 64)
        sd.paged4_attention(*args, **kw, out=got, workspace=ws)
        sd.sdpa_forward(q, q, q, outs[1], 2, 4, 512, 512, 64, 64)

    for _ in range(5):
        run()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(x, other) for x in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for x in (got, *outs):
        x.zero_()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(x, other) for x in outs)
    sd.sdpa_device_check()


def test_bad_pages_are_reported_and_read_as_zeros():
    rng = np.random.default_rng(4504)
    for bad in (-1, 10 ** 6, -7):
        c = _case(rng, [150, 2], [400, 90], 4, 2, 64, 16)
        c["cache"].table[0, 3] = bad
        for held in c["held"]:
            held[0][48:64] = 0.0
        got = sd.paged4_attention(*_args(c), **_kw(c))
        with pytest.raises(sd.SdpaError) as e:
            sd.sdpa_device_check()
        assert e.value.status == 7
        _check(got, c)


def test_a_page_of_more_than_32_bits():
    """One page of 2^25 positions of 256 columns, 4.5 GB for keys and as much for
    values: the last positions appended, read and attended to through a window."""
    import torch
    rng = np.random.default_rng(4505)
    d, page, window, sinks = 256, 1 << 25, 300, 4
    kp, vp = (torch.zeros((1, 1, page, 9 * d // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = dev_int(np.zeros((1, 1), np.int32))
    held = [np.zeros((0, 1, d)) for _ in range(2)]
    for new, length in ((10, 10), (900, page - 1), (1, page)):
        k, v = (_bf16(rng, (new, 1, d)) for _ in range(2))
        starts, lens = dev_int(pu.starts_of([new])), dev_int([length])
        sd.paged4_append(None, dev(k), dev(v), kp, vp, table, starts, lens)
        now = [p4.values(*p4.quantise(x)) for x in (k, v)]
        out = [torch.empty(new, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sd.paged4_read(kp, vp, table, starts, lens, *out)
        assert all(np.array_equal(host(x), y) for x, y in zip(out, now))
        held = [np.concatenate((x, y)) for x, y in zip(held, now)]
    for new in (1, 60):
        q = _bf16(rng, (new, 2, d))
        got = host(sd.paged4_attention(dev(q), kp, vp, table, dev_int(pu.starts_of([new])), dev_int([page]),
                                       window=window, sinks=sinks))
        # the first 10 positions and the last 901, as a sequence of 911: the window hides the seam
        ref, bound = p4.attention(q, [held[0]], [held[1]], pu.starts_of([new]), [911], 0.0, window, sinks)
        assert np.all(np.abs(got - ref) <= bound)
    sd.sdpa_device_check()


def test_read_of_many_tokens():
    """Blocks of tokens over many short sequences, rows that are no sequence's before
    and behind them, negative positions and bad pages among them."""
    rng = np.random.default_rng(4506)
    h_kv, d, page, first, behind = 3, 64, 16, 37, 50
    lens = [int(x) for x in rng.integers(0, 70, size=400)]
    new = [int(rng.integers(0, n + 8)) for n in lens]
    cache = pu.Cache(rng, lens, h_kv, d, page)
    dense = [[_bf16(rng, (n, h_kv, d)) for n in lens] for _ in range(2)]
    made = [p4.pages_of(cache, x, 0xFF, 0) for x in dense]
    bad = int(np.argmax(lens))
    new[bad] = lens[bad]
    cache.table[bad, 1] = -1
    starts = pu.starts_of(new, first)
    t = int(starts[-1]) + behind
    assert t > 16 * 160
    out = _read(cache, [_bytes(m[0]) for m in made], starts, t, (0, 0))
    with pytest.raises(sd.SdpaError):
        sd.sdpa_device_check()
    for got, (_, held) in zip(out, made):
        held[bad][page:2 * page] = 0.0
        for s, n in enumerate(new):
            rows = got[starts[s]:starts[s + 1]]
            want = np.zeros((n, h_kv, d))
            if min(n, lens[s]):
                want[n - min(n, lens[s]):] = held[s][lens[s] - min(n, lens[s]):]
            assert np.array_equal(rows, want), s
    # (_read fills what it hands out with a value first)
    untouched = _read(cache, [_bytes(m[0]) for m in made], pu.starts_of([0] * 400), t, (0, 0))
    for got, before in zip(out, untouched):
        assert np.array_equal(got[:first], before[:first]) and np.array_equal(got[int(starts[-1]):], before[int(starts[-1]):])


@pytest.fixture(scope="module")
def faulty_lib():
    """A copy of the library whose kernel for many rows never signals a unit's first scores."""
    sd_build.build()
    d = tempfile.mkdtemp(prefix="sdpa_paged4_test_")
    nvcc = sd_build._nvcc()
    obj = os.path.join(d, "paged4_test.o")
    subprocess.check_call([nvcc] + sd_build._flags() + ["-DSDPA_TEST_WITHHOLD_FIRST_S_COMMIT",
                                                        "-DSDPA_TEST_WAIT_LIMIT=200000000ll", "-c",
                                                        os.path.join(sd_build.CSRC, "paged4_wide.cu"), "-o", obj])
    others = [os.path.join(sd_build.BUILD_DIR, s.replace(".cu", ".o")) for s in sd_build.SOURCES if s != "paged4_wide.cu"]
    path = os.path.join(d, "libsdpa_paged4_test.so")
    subprocess.check_call([nvcc] + sd_build.ARCH + ["-shared", "-cudart", "static", "-o", path, obj] + others)
    return sd.load_library(path)


@pytest.mark.parametrize("d", [64, 256])
def test_bounded_waits_time_out_and_report(faulty_lib, d):
    import torch
    rng = np.random.default_rng(4600)
    c = _case(rng, [200, 1], [5000, 400], 8, 2, d, 32)
    args = _args(c)
    ws = sd.paged4_workspace(args[0], args[1], args[3])
    out = torch.zeros_like(args[0])
    t0 = time.time()
    rc = faulty_lib.sdpa_paged4_forward(
        args[0].data_ptr(), args[1].data_ptr(), args[2].data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), 2, 201, 8,
        2, d, 32, c["cache"].n_pages, c["cache"].per_seq, args[3].data_ptr(), args[4].data_ptr(), args[5].data_ptr(),
        8 * d, ctypes.c_float(0.0), *c["exps"], 0, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert faulty_lib.sdpa_device_check() == 6                   # SDPA_ERR_DEVICE_TIMEOUT
    assert time.time() - t0 < 30.0
    assert faulty_lib.sdpa_device_check() == 0                   # cleared
    # the product library computes the right answer, in the same workspace
    got = sd.paged4_attention(*args, **_kw(c), workspace=ws)
    sd.sdpa_device_check()
    _check(got, c)
