"""What the scores of the attention over the cache in 4 bits go through, in the kernel
for few rows (sequences of up to 32 rows a key-value head) and the one for many:
ranges of queries, units and scales whose product is ordinary.  Against the plain fp64 implementation and bounds of paged4_util.py."""
import numpy as np
import pytest

from test_gpu_paged4 import _case, _check, _run

pytestmark = pytest.mark.gpu

ROWS = {"few": ([3, 1], [50, 700]), "many": ([200, 1], [500, 700])}


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("k_std,q_by,scale,k_exp", [
    # queries of 2^112: 2^99 with 2^32 is no float, the whole product is 2^-16
    (2.0 ** 32, 2.0 ** 80, 2.0 ** -147, 32),
    # and of 2^-108: 2^-120 with 2^-32 is no float, the whole product is 2^-25
    (2.0 ** -23, 2.0 ** -85, 2.0 ** 127, -32),
    # the scale is no whole power of two, and below the ordinary floats
    (2.0 ** 30, 2.0 ** 78, 1.25 * 2.0 ** -143, 32)])
def test_ranges_that_only_the_whole_product_fits(rows, d, k_std, q_by, scale, k_exp):
    rng = np.random.default_rng(4800 + d)
    # (queries like keys of k_std, and q_by times that; a row of zeros, keys of zeros)
    c = _case(rng, *ROWS[rows], 4, 2, d, 16, std=k_std, exps=(k_exp, -3))
    c["q"] = (c["q"] * np.float32(q_by)).astype(np.float32)
    c["q"][1, 2] = 0.0
    scale = float(np.float32(scale / np.sqrt(d / 64)))
    _check(_run(c, scale=scale), c, scale)
