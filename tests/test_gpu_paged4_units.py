"""Attention over the cache in 4 bits where every run of the kernel for many rows
takes several units, whole and one after another: a warp that has stored a unit's
rows is at the next unit's while the others of its 128 rows may not be.  Against the
plain fp64 implementation and bounds of paged4_util.py, and again and again."""
import numpy as np
import pytest

import paged4_util as p4
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import host
from test_gpu_paged4 import _args, _case, _kw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_whole_units(d):
    """64 sequences of 16 key-value heads, more than 128 rows each, on 152 runs."""
    import torch
    rng = np.random.default_rng(4700 + d)
    new = [int(x) for x in rng.integers(129, 200, size=64)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 150, size=64))]
    c = _case(rng, new, lens, 16, 16, d, 32)
    args, kw = _args(c), _kw(c)
    ws = sd.paged4_workspace(args[0], args[1], args[3])
    want = sd.paged4_attention(*args, **kw, workspace=ws)
    outs = [torch.empty_like(want) for _ in range(10)]
    for _ in range(3):
        for out in outs:
            sd.paged4_attention(*args, **kw, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in outs)
    sd.sdpa_device_check()
    got, starts = host(want), c["starts"]
    for s in range(0, 64, 7):
        rows = slice(int(starts[s]), int(starts[s + 1]))
        ref, bound = p4.attention(c["q"][rows], [c["held"][0][s]], [c["held"][1][s]], [0, new[s]], [lens[s]])
        assert np.all(np.abs(got[rows] - ref) <= bound), s
