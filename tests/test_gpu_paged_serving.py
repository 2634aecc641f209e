"""Rotation on the way into the cache, step by step: what the append returns
and stores is the rotation of the very rows that it was given, within the
rotation's own bound (paged_util.py), in a serving loop and in pages whose
offsets pass 32 bits."""
import numpy as np
import pytest

import paged_util as pu
import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int, host
from test_gpu_paged import _bf16, _Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("schedule", [[[90, 33, 1]], [[40, 1, 0], [7, 30, 1], [43, 2, 0]],
                                      [[80, 20, 0]] + [[1, 1, 1]] * 13], ids=["whole", "chunks", "tokens"])
def test_every_step_stores_the_rotation_of_its_own_projection(schedule):
    lens, h, h_kv, d, dm, page = [90, 33, 1], 8, 2, 64, 256, 16
    rng = np.random.default_rng(810)
    cache = pu.Cache(rng, lens, h_kv, d, page)
    layer = _Layer(rng, cache, h, h_kv, d, dm, sum(lens))
    freqs = pu.freqs_of(d)
    done = [0] * len(lens)
    kept = {}                                                   # (sequence, position): key and value as stored
    for chunk in schedule:
        new = [min(c, n - a) for c, n, a in zip(chunk, lens, done)]
        done = [a + n for a, n in zip(done, new)]
        starts, t = pu.starts_of(new), sum(new)
        layer.step(dev(_bf16(rng, (t, dm))), dev_int(starts), dev_int(np.array(done, np.int32)))
        sd.sdpa_device_check()
        rows = host(layer.qkv).reshape(-1, h + 2 * h_kv, d)[:t]
        where = pu.positions_of(t, starts, done)
        want, bound = pu.rotate(rows[:, :h + h_kv], np.array(where), freqs, False)
        assert np.all(np.abs(host(layer.q)[:t] - want[:, :h]) <= bound[:, :h])
        kp, vp = host(layer.kp), host(layer.vp)
        for s in range(len(lens)):
            for i in range(starts[s], starts[s + 1]):
                at = (cache.table[s, where[i] // page], slice(None), where[i] % page)
                assert np.all(np.abs(kp[at] - want[i, h:]) <= bound[i, h:])
                assert np.array_equal(vp[at], rows[i, h + h_kv:])
                kept[s, where[i]] = (at, kp[at], vp[at])
        for at, k, v in kept.values():                          # earlier steps' rows stay
            assert np.array_equal(kp[at], k) and np.array_equal(vp[at], v)
    assert done == lens and len(kept) == sum(lens)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_pages_hold_rotated_keys(interleaved):
    """Pages whose element offsets pass 32 bits, filled with rotation and read."""
    import torch
    h_kv, page, d = 8, 256, 128
    n_pages = (1 << 32) // (h_kv * page * d) + 3
    rng = np.random.default_rng(811)
    kp = torch.empty((n_pages, h_kv, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = np.array([[n_pages - 1, 0], [n_pages - 2, n_pages // 2 + 1]], np.int32)
    lens = np.array([300, 400], np.int32)
    k, v = ([_bf16(rng, (n, h_kv, d)) for n in lens] for _ in range(2))
    freqs = pu.freqs_of(d)
    tab, ln = dev_int(table), dev_int(lens)
    sd.paged_append(None, dev(np.concatenate(k)), dev(np.concatenate(v)), kp, vp, tab, dev_int(pu.starts_of(lens)), ln,
                    dev(freqs, "f32"), interleaved)
    sd.sdpa_device_check()
    stored = []
    for s, n in enumerate(lens):
        want, bound = pu.rotate(k[s], np.arange(n), freqs, interleaved)
        got = [np.concatenate([host(pages[int(x)]).transpose(1, 0, 2) for x in table[s]])[:n] for pages in (kp, vp)]
        assert np.all(np.abs(got[0] - want) <= bound)
        assert np.array_equal(got[1], v[s])
        stored.append(got[0])
    starts = pu.starts_of([2, 1])
    q = _bf16(rng, (3, h_kv, d))
    got = host(sd.paged_attention(dev(q), kp, vp, tab, dev_int(starts), ln))
    sd.sdpa_device_check()
    ref, bound = pu.attention(q, stored, v, starts, lens)
    assert np.all(np.abs(got - ref) <= bound)
