"""The append's angles at far positions.  Pairs (a, b) are chosen so that the
rotated value nearly cancels: its own rounding is far below what an error of
the angle moves it by, |(a, b)| times the error.  The angle is worked out in
whole numbers (position times the fp32 frequency, divided by 2 pi to 200 bits),
since 64 bits lose it too: a product of 30 and 24 bits is rounded by up to
2^-54 of itself, 1e-5 rad at 2^30 positions and 100 rad a position."""
import numpy as np
import pytest

import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int, host

pytestmark = pytest.mark.gpu

BITS = 200


def _arctan_of_inverse(n, one):
    total, term, k = 0, one // n, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


def _inverse_of_two_pi():
    """2^BITS / (2 pi), with Machin's formula for pi."""
    one = 1 << (BITS + 64)
    pi = 4 * (4 * _arctan_of_inverse(5, one) - _arctan_of_inverse(239, one))
    return (one << BITS) // (2 * pi)


def _angles(positions, freqs):
    """[positions, freqs] angles in (-pi, pi], each good to fp64's rounding."""
    inverse = _inverse_of_two_pi()
    out = np.empty((len(positions), len(freqs)))
    for j, f in enumerate(freqs):
        m, e = np.frexp(np.float64(f))
        m, e = int(m * 2 ** 24), int(e) - 24                    # f = m 2^e
        shift = BITS - e
        for i, p in enumerate(positions):
            turns = int(p) * m * inverse % (1 << shift)
            if turns >> (shift - 1):
                turns -= 1 << shift
            out[i, j] = turns / (1 << shift) * 2 * np.pi
    return out


def _bf16(x):
    return synthetic.round_to_bf16(np.asarray(x, np.float32)).astype(np.float64)


def _cancelling(t):
    """bf16 (a, b) with a cos t - b sin t as near to zero as 128 choices give."""
    c, s = np.cos(t)[..., None], np.sin(t)[..., None]
    one = np.arange(128, 256, dtype=np.float64) / 128           # every bf16 value from 1 to 2
    steep = np.abs(s) > np.abs(c)
    a = np.where(steep, one, _bf16(one * np.divide(s, c, out=np.zeros_like(s), where=~steep)))
    b = np.where(steep, _bf16(one * np.divide(c, s, out=np.zeros_like(c), where=steep)), one)
    best = np.argmin(np.abs(a * c - b * s), axis=-1)[..., None]
    return np.take_along_axis(a, best, -1)[..., 0], np.take_along_axis(b, best, -1)[..., 0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [1.0, 100.0, 1e4])
@pytest.mark.parametrize("log_position", [10, 17, 24, 29, 30])
def test_append_angles(log_position, top, interleaved):
    import torch
    rng = np.random.default_rng(900 + log_position)
    d, page, b = 128, 1 << 20, 40
    per_seq = min(1 << max(log_position - 20, 0), 1023)         # 2^30 positions are too many by one page
    slots = rng.choice(1 << min(log_position, 20), size=b, replace=False)
    positions = slots + (rng.integers(per_seq // 2, per_seq, size=b) << 20 if per_seq > 1 else 0)
    positions[0] = min(1 << log_position, per_seq * page) - 1   # the last one
    slots = positions % page
    keep = np.unique(slots, return_index=True)[1]               # each token has a slot of its own
    positions, slots = positions[keep], slots[keep]
    b = len(positions)
    freqs = np.geomspace(top, top * 1e-5, d // 2).astype(np.float32)
    t = _angles(positions, freqs)
    x0, x1 = _cancelling(t)
    lo, hi = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    rows = np.empty((b, 1, d), np.float32)
    rows[:, 0, lo], rows[:, 0, hi] = x0, x1
    kp = torch.zeros((1, 1, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    x = dev(rows)
    q_out = sd.paged_append(x, x, x, kp, vp, dev_int(np.zeros((b, per_seq), np.int32)),
                            dev_int(np.arange(b + 1, dtype=np.int32)), dev_int((positions + 1).astype(np.int32)),
                            dev(freqs, "f32"), interleaved)
    sd.sdpa_device_check()
    want = np.empty((b, 1, d))
    want[:, 0, lo], want[:, 0, hi] = x0 * np.cos(t) - x1 * np.sin(t), x1 * np.cos(t) + x0 * np.sin(t)
    size = np.empty((b, 1, d))
    size[:, 0, lo] = size[:, 0, hi] = np.abs(x0) + np.abs(x1)
    assert np.median(np.abs(want[:, 0, lo])) < 2.0 ** -13       # they do cancel: 2^-21 is rounded off at most
    # pu.rotate's bound: a bf16 rounding, and 2.2e-6 (|a| + |b|) rounded along
    bound = (2.0 ** -8 * np.abs(want) + 2.2e-6 * size) * (1 + 2.0 ** -8)
    assert np.all(np.abs(host(q_out) - want) <= bound)
    assert np.all(np.abs(host(kp)[0, 0, slots][:, None] - want) <= bound)
    assert np.array_equal(host(vp)[0, 0, slots][:, None], rows)
