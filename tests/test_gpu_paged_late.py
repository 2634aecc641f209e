"""Pieces that come late in the paged attention: a copy of its kernel, compiled
here so that waits inside a CTA give up after 20 million clock cycles and runs
publish 100 million late (about 50 ms), still computes the same: waits for other
runs' pieces may take longer by so much for each item of a run, here 400000
cycles.  (test_gpu_paged_timeout.py has waits that run out.)"""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest

import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from transformer_scaled_dot_02_gb300 import build as sd_build
from gpu_util import dev, dev_int

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def late_lib():
    """A copy of the library whose paged kernels wait less and publish late."""
    sd_build.build()
    d = tempfile.mkdtemp(prefix="sdpa_paged_late_")
    nvcc = sd_build._nvcc()
    obj = os.path.join(d, "paged_late.o")
    subprocess.check_call([nvcc] + sd_build._flags() + ["-DSDPA_TEST_WAIT_LIMIT=20000000ll",
                                                        "-DSDPA_TEST_ITEM_CYCLES=400000ll",
                                                        "-DSDPA_TEST_LATE_PUBLISH=100000000ll", "-c",
                                                        os.path.join(sd_build.CSRC, "paged.cu"), "-o", obj])
    others = [os.path.join(sd_build.BUILD_DIR, s.replace(".cu", ".o")) for s in sd_build.SOURCES if s != "paged.cu"]
    lib_path = os.path.join(d, "libsdpa_paged_late.so")
    subprocess.check_call([nvcc] + sd_build.ARCH + ["-shared", "-cudart", "static", "-o", lib_path, obj] + others)
    return sd.load_library(lib_path)


# Units of one head whose 304 runs (two for each of 152 SMs) have 1000 items, quarters
# of a key tile, and more: so each may wait 400 million cycles beyond the 20 million.
# 60 units are cut into 5 or 6 pieces, which the last run merges alone, 15 into 20
# and more, which go in slices.
@pytest.mark.parametrize("new", [17, 1], ids=["wide", "narrow"])
@pytest.mark.parametrize("b,h_kv,length", [(15, 4, 84000), (15, 1, 340000)], ids=["together", "slices"])
def test_runs_wait_for_pieces_that_come_late(late_lib, b, h_kv, length, new):
    import torch
    d, page = 64, 64
    rng = np.random.default_rng(5)
    need = -(-length // page)
    table = np.tile(rng.permutation(need).astype(np.int32), (b, 1))          # every sequence reads the same pages
    kp, vp = (torch.randn((need, h_kv, page, d), generator=torch.Generator("cuda").manual_seed(s), device="cuda",
                          dtype=torch.bfloat16) for s in (1, 2))
    q = dev(synthetic.round_to_bf16(rng.standard_normal((b * new, h_kv, d)).astype(np.float32)))
    lens = np.full(b, length, np.int32) - 64 * np.arange(b, dtype=np.int32)
    args = (q, kp, vp, dev_int(table), dev_int(pu.starts_of([new] * b)), dev_int(lens))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert int(lens.sum()) // 64 * h_kv * 4 >= 1000 * 2 * sms
    ws = sd.paged_workspace(q, kp, args[3])
    want = sd.paged_attention(*args, workspace=ws)
    sd.sdpa_device_check()
    for _ in range(2):
        out = torch.full_like(q, float("nan"))
        rc = late_lib.sdpa_paged_forward(
            q.data_ptr(), kp.data_ptr(), vp.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), b, b * new, h_kv,
            h_kv, d, page, need, need, args[3].data_ptr(), args[4].data_ptr(), args[5].data_ptr(), h_kv * d,
            ctypes.c_float(0.0), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert late_lib.sdpa_device_check() == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
