"""Failure detection in the paged attention without a GPU fault: a copy of its
kernel, compiled here so that a CTA's first score tile is never signalled,
gives up its bounded waits (those on other CTAs' pieces among them), reports a
timeout and leaves the context usable.  Another copy, whose CTAs do not wait for
pieces of later ones, still computes the same."""
import ctypes
import os
import subprocess
import tempfile
import time

import numpy as np
import pytest

import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from transformer_scaled_dot_02_gb300 import build as sd_build
from gpu_util import dev, dev_int, host

pytestmark = pytest.mark.gpu


def _library(define):
    """A copy of the library whose paged kernels are compiled with `define`."""
    sd_build.build()
    d = tempfile.mkdtemp(prefix="sdpa_paged_test_")
    nvcc = sd_build._nvcc()
    obj = os.path.join(d, "paged_test.o")
    subprocess.check_call([nvcc] + sd_build._flags() + ["-D" + define, "-c",
                                                        os.path.join(sd_build.CSRC, "paged.cu"), "-o", obj])
    others = [os.path.join(sd_build.BUILD_DIR, s.replace(".cu", ".o")) for s in sd_build.SOURCES if s != "paged.cu"]
    lib_path = os.path.join(d, "libsdpa_paged_test.so")
    subprocess.check_call([nvcc] + sd_build.ARCH + ["-shared", "-cudart", "static", "-o", lib_path, obj] + others)
    return sd.load_library(lib_path)


@pytest.fixture(scope="module")
def faulty_lib():
    return _library("SDPA_TEST_WITHHOLD_FIRST_S_COMMIT")


@pytest.fixture(scope="module")
def impatient_lib():
    return _library("SDPA_TEST_PATIENCE=-1")


@pytest.mark.parametrize("new,length", [(1, 1000), (40, 900)])
def test_bounded_waits_time_out_and_report(faulty_lib, new, length):
    import torch
    rng = np.random.default_rng(3)
    h, h_kv, d = 8, 2, 64
    bf16 = lambda shape: synthetic.round_to_bf16(rng.standard_normal(shape).astype(np.float32))
    cache = pu.Cache(rng, [length], h_kv, d, 32)
    k, v = [bf16((length, h_kv, d))], [bf16((length, h_kv, d))]
    kp, vp = dev(cache.pages_of(k, 0.0)), dev(cache.pages_of(v, 0.0))
    q, starts = bf16((new, h, d)), np.array([0, new], np.int32)
    args = (dev(q), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    ws = sd.paged_workspace(args[0], kp, args[3])
    out = torch.zeros_like(args[0])
    t0 = time.time()
    rc = faulty_lib.sdpa_paged_forward(
        args[0].data_ptr(), kp.data_ptr(), vp.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), 1, new, h, h_kv,
        d, 32, cache.n_pages, cache.per_seq, args[3].data_ptr(), args[4].data_ptr(), args[5].data_ptr(), h * d,
        ctypes.c_float(0.0), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert faulty_lib.sdpa_device_check() == 6                   # SDPA_ERR_DEVICE_TIMEOUT
    assert time.time() - t0 < 30.0
    assert faulty_lib.sdpa_device_check() == 0                   # cleared
    # the product library computes the right answer, in the same workspace
    got = host(sd.paged_attention(*args, workspace=ws))
    sd.sdpa_device_check()
    ref, bound = pu.attention(q, k, v, starts, cache.lens)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("h,h_kv,d,new,lens", [(2, 2, 64, [69], [26595]), (16, 1, 64, [1, 1], [33000, 20000]),
                                               (16, 4, 64, [1, 1], [70000, 300]), (1, 1, 128, [1], [40000])])
def test_slices_that_are_left_fall_to_the_last_run(impatient_lib, h, h_kv, d, new, lens):
    """Runs that do not wait for the others' pieces leave their slices to the
    unit's last run; the slices are the same ones, so the bits are too."""
    import torch
    rng = np.random.default_rng(4)
    bf16 = lambda shape: synthetic.round_to_bf16(rng.standard_normal(shape).astype(np.float32))
    cache = pu.Cache(rng, lens, h_kv, d, 64)
    kp, vp = (dev(cache.pages_of([bf16((n, h_kv, d)) for n in lens], 0.0)) for _ in range(2))
    starts = pu.starts_of(new)
    args = (dev(bf16((sum(new), h, d))), kp, vp, dev_int(cache.table), dev_int(starts), dev_int(cache.lens))
    ws = sd.paged_workspace(args[0], kp, args[3])
    want = sd.paged_attention(*args, workspace=ws)
    for _ in range(4):
        out = torch.full_like(args[0], float("nan"))
        rc = impatient_lib.sdpa_paged_forward(
            args[0].data_ptr(), kp.data_ptr(), vp.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), len(lens),
            sum(new), h, h_kv, d, 64, cache.n_pages, cache.per_seq, args[3].data_ptr(), args[4].data_ptr(),
            args[5].data_ptr(), h * d, ctypes.c_float(0.0), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and impatient_lib.sdpa_device_check() == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    sd.sdpa_device_check()
