"""What the scores and weights of the attention over the cache in 4 bits go through,
in the kernel for few rows (sequences of up to 32 rows a key-value head) and the one
for many: units of keys, ranges of queries, units and scales whose product is
ordinary, weak keys behind strong ones, scores of many bits.  Against the plain fp64
implementation and bounds of paged4_util.py."""
import numpy as np
import pytest

import paged4_util as p4
from gpu_util import host
from test_gpu_paged4 import _bf16, _case, _check, _run

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
    # (queries like keys of k_std, and q_by times that; a row of zeros)
    c = _case(rng, *ROWS[rows], 4, 2, d, 16, std=k_std, exps=(k_exp, -3))
    c["q"] = (c["q"] * np.float32(q_by)).astype(np.float32)
    c["q"][1, 2] = 0.0
    scale = float(np.float32(scale / np.sqrt(d / 64)))
    _check(_run(c, scale=scale), c, scale)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", [16, 64, 128, 256])
@pytest.mark.parametrize("k_exp", [-3, 5])
def test_units_of_keys(rows, d, k_exp):
    rng = np.random.default_rng(4810 + d + k_exp)
    c = _case(rng, *ROWS[rows], 6, 2, d, 32, exps=(k_exp, 2), window=300, sinks=5)
    _check(_run(c), c)


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
def test_weak_keys_behind_a_strong_one_count(rows, d):
    """The first key of a sequence has nearly all of the weight, and every other one
    2^-25.6 of its: their values are all that the output has.  A weight is rounded to
    fp16 at 2^5 times itself: off by 2^-11 of itself, or, where that is below 2^-14, by
    half of fp16's smallest step, 2^-25 / 2^5 = 2^-30."""
    new, n = (2, 511) if rows == "few" else (200, 900)
    rng = np.random.default_rng(4820 + d)
    c = _case(rng, [new], [n], 2, 1, d, 32, exps=(0, 0))
    k, v = np.zeros((n, 1, d), np.float32), np.ones((n, 1, d), np.float32)
    k[:, 0, 0], k[0, 0, 0] = -6.0, 6.0
    v[0] = 0.0
    v[:, 0, ::16] = 6.0
    v[0] = 0.0
    made = [p4.pages_of(c["cache"], [x], 0xFF, 0) for x in (k, v)]
    q = np.zeros((new, 2, d), np.float32)
    q[..., 0] = 1.0
    c.update(pages=[m[0] for m in made], held=[m[1] for m in made], q=q)
    assert np.array_equal(c["held"][0][0], k) and np.array_equal(c["held"][1][0], v)
    scale = float(np.float32(25.6 / 12.0 * np.log(2.0)))
    got = host(_run(c, scale=scale))
    for i in range(new):
        weak = np.float64(n - new + i) * np.exp(-12.0 * scale)
        want = weak / (1.0 + weak) * v[1, 0]
        # fp32 scores and sums as in paged4_util: e = d 2^-23 scale 6
        share = 2.0 ** -11 + 2.1 * d * 2.0 ** -23 * scale * 6.0 + 2.0 ** -14 + 2.0 ** -8
        bound = (share * want + 2.0 ** -30 * (n - new + i) * v[1, 0]) * (1 + 2.0 ** -8)
        assert np.all(np.abs(got[i] - want) <= bound), (i, got[i, 0, :2], want[:2], bound[:2])


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
@pytest.mark.parametrize("log_q", [1, 17, 20, 22])
def test_scores_of_many_bits(rows, d, log_q):
    """Scores up to 2^25.9, in fp32 exact but for the scale: those of one key are 5 (7.2 in
    log2 units) above all others', which begins to count a tile after the first.
    What is left of a score less a maximum is small, and off by fp32's half step of it
    and by 2^-24 of the difference (the scale's rounding): 2^-20 of a weight in all."""
    new, n = (9, 300) if rows == "few" else (130, 700)
    rng = np.random.default_rng(4830 + d)
    c = _case(rng, [new], [n], 3, 1, d, 16, exps=(0, 0))
    k, v = np.zeros((n, 1, d), np.float32), _bf16(rng, (n, 1, d))
    k[:, 0, 0] = 6.0
    k[150, 0, 1] = 4.0
    held_v = p4.values(*p4.quantise(v))
    made = p4.pages_of(c["cache"], [k], 0xFF, 0), p4.pages_of(c["cache"], [v], 0xFF, 0)
    q = np.zeros((new, 3, d), np.float32)
    # seven bits below the first: maxima of all kinds of rounding
    q[..., 0] = (1.0 + 5 * np.arange(new * 3).reshape(new, 3) % 128 / 128.0) * 2.0 ** log_q
    q[..., 1] = 1.0
    c.update(pages=[m[0] for m in made], held=[m[1] for m in made], q=q)
    got = host(_run(c, scale=1.25))
    for i in range(new):
        seen = n - new + i + 1
        w = np.ones(seen)
        w[150] = np.exp(5.0)
        w /= w.sum()
        want, mass, total = w @ held_v[:seen, 0], w @ np.abs(held_v[:seen, 0]), np.abs(held_v[:seen, 0]).sum(0)
        bound = ((2.0 ** -11 + 2.0 ** -20 + 2.0 ** -14) * mass + 2.0 ** -30 * total + 2.0 ** -8 * np.abs(want)) * (1 + 2.0 ** -8)
        assert np.all(np.abs(got[i] - want) <= bound), i
