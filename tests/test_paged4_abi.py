"""The entry points of the cache in 4 bits on the CPU: argument checks return
their documented codes, the workspace size follows the shapes, the helpers refuse
what the entry points cannot see, and the fp64 reference that the GPU tests use
agrees with a plain search for the nearest numbers."""
import ctypes

import numpy as np
import pytest

import paged4_util as p4
import transformer_scaled_dot_02_gb300 as sd
from transformer_scaled_dot_02_gb300 import build as sd_build

INVALID, UNSUPPORTED, NODEV, WORKSPACE = 1, 2, 3, 4
A, MIS = 1 << 40, (1 << 40) + 8       # placeholder addresses: no call below reaches CUDA work
STEP = 1 << 32


def _gpu_visible():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


@pytest.fixture(scope="module")
def lib():
    sd_build.build()
    return sd.load_library()


SHAPE = dict(b=3, t=5, h=8, h_kv=2, d=64, page=16, n_pages=40, per_seq=12, table=A, starts=A, lens=A, kp=A,
             vp=A + STEP, ke=0, ve=-3)


def _append(lib, **kw):
    a = dict(SHAPE, q=A + 2 * STEP, k=A + 3 * STEP, v=A + 4 * STEP, q_out=A + 5 * STEP, qs=512, ks=128, vs=128,
             freqs=A, d_rot=64, inter=0)
    a.update(kw)
    return lib.sdpa_paged4_append(a["q"], a["k"], a["v"], a["q_out"], a["kp"], a["vp"], a["b"], a["t"], a["h"],
                                  a["h_kv"], a["d"], a["page"], a["n_pages"], a["per_seq"], a["table"], a["starts"],
                                  a["lens"], a["qs"], a["ks"], a["vs"], a["freqs"], a["d_rot"], a["inter"], a["ke"],
                                  a["ve"], None)


def _read(lib, **kw):
    a = dict(SHAPE, ko=A + 2 * STEP, vo=A + 3 * STEP)
    a.update(kw)
    a["h_kv"] = a["h"] if "h" in kw else a["h_kv"]
    return lib.sdpa_paged4_read(a["kp"], a["vp"], a["ko"], a["vo"], a["b"], a["t"], a["h_kv"], a["d"], a["page"],
                                a["n_pages"], a["per_seq"], a["table"], a["starts"], a["lens"], a["ke"], a["ve"], None)


def _forward(lib, **kw):
    a = dict(SHAPE, q=A + 2 * STEP, out=A + 3 * STEP, ws=A + 4 * STEP, ws_bytes=1 << 40, qs=512, scale=0.0, window=0,
             sinks=0)
    a.update(kw)
    return lib.sdpa_paged4_forward(a["q"], a["kp"], a["vp"], a["out"], a["ws"], a["ws_bytes"], a["b"], a["t"], a["h"],
                                   a["h_kv"], a["d"], a["page"], a["n_pages"], a["per_seq"], a["table"], a["starts"],
                                   a["lens"], a["qs"], ctypes.c_float(a["scale"]), a["ke"], a["ve"], a["window"],
                                   a["sinks"], None)


CALLS = [_append, _read, _forward]


@pytest.mark.parametrize("call", CALLS)
def test_shared_argument_checks(lib, call):
    for name in ("kp", "vp", "table", "starts", "lens"):
        assert call(lib, **{name: None}) == INVALID, name
        assert call(lib, **{name: A + 2}) == INVALID, name
    assert call(lib, kp=MIS) == INVALID and call(lib, vp=MIS) == INVALID
    for name in ("b", "d", "page", "n_pages", "per_seq", "h_kv"):
        assert call(lib, **{name: 0}) == INVALID, name
    assert call(lib, t=-1) == INVALID
    for d in (8, 48, 80, 512):
        assert call(lib, d=d, qs=8 * d, ks=2 * d, vs=2 * d, d_rot=0) == UNSUPPORTED if call is _append else \
            call(lib, d=d, **({"qs": 8 * d} if call is _forward else {})) == UNSUPPORTED
    for page in (8, 24, 1000):
        assert call(lib, page=page) == UNSUPPORTED
    assert call(lib, per_seq=1 << 27) == UNSUPPORTED
    for e in (33, -33, 1 << 30, -(1 << 31)):
        assert call(lib, ke=e) == UNSUPPORTED and call(lib, ve=e) == UNSUPPORTED


def test_append_checks(lib):
    for name in ("k", "v", "q", "q_out"):
        assert _append(lib, **{name: None}) == INVALID, name
        assert _append(lib, **{name: MIS + STEP * 7}) == INVALID, name
    assert _append(lib, h=7) == INVALID
    assert _append(lib, h=2 * 129, qs=2 * 129 * 64) == UNSUPPORTED
    assert _append(lib, qs=511) == INVALID and _append(lib, ks=120) == INVALID and _append(lib, vs=64) == INVALID
    assert _append(lib, qs=516) == UNSUPPORTED and _append(lib, ks=132) == UNSUPPORTED
    assert _append(lib, d_rot=80) == INVALID and _append(lib, d_rot=-16) == INVALID
    assert _append(lib, d_rot=24) == UNSUPPORTED
    assert _append(lib, freqs=None) == INVALID and _append(lib, freqs=A + 1) == INVALID
    # rows and pages that share memory
    assert _append(lib, q_out=A + 2 * STEP, qs=1024) == INVALID
    assert _append(lib, q_out=A + 3 * STEP) == INVALID and _append(lib, q_out=A + 4 * STEP + 16) == INVALID
    assert _append(lib, vp=A + 16) == INVALID
    for name in ("q", "k", "v", "q_out"):
        assert _append(lib, **{name: A + 64}) == INVALID and _append(lib, **{name: A + STEP + 64}) == INVALID, name


def test_read_checks(lib):
    for name in ("ko", "vo"):
        assert _read(lib, **{name: None}) == INVALID
        assert _read(lib, **{name: MIS + STEP * 7}) == INVALID
        assert _read(lib, **{name: A + 64}) == INVALID and _read(lib, **{name: A + STEP + 64}) == INVALID
    assert _read(lib, vo=A + 2 * STEP + 16) == INVALID


def test_forward_checks(lib):
    for name in ("q", "out"):
        assert _forward(lib, **{name: None}) == INVALID
        assert _forward(lib, **{name: MIS + STEP * 7}) == INVALID
    assert _forward(lib, h=7) == INVALID
    assert _forward(lib, out=A + 2 * STEP) == INVALID and _forward(lib, out=A + 64) == INVALID
    assert _forward(lib, qs=511) == INVALID and _forward(lib, qs=516) == UNSUPPORTED
    for scale in (-1.0, float("inf"), float("nan")):
        assert _forward(lib, scale=scale) == INVALID
    assert _forward(lib, window=-1) == INVALID and _forward(lib, sinks=-1) == INVALID
    assert _forward(lib, ws=None, per_seq=4096) == WORKSPACE
    assert _forward(lib, ws=MIS, per_seq=4096) == WORKSPACE
    need = sd.sdpa_paged4_workspace_size(3, 5, 8, 2, 64, 16, 4096)
    assert need > 0 and _forward(lib, ws_bytes=need - 1, per_seq=4096) == WORKSPACE


@pytest.mark.skipif(_gpu_visible(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("call", CALLS)
def test_valid_arguments_reach_the_device_check(lib, call):
    assert call(lib) == NODEV
    assert call(lib, t=0) == NODEV
    if call is _forward:
        assert call(lib, window=1, sinks=1 << 30) == NODEV and call(lib, window=(1 << 31) - 1) == NODEV


def test_workspace_size(lib):
    size = sd.sdpa_paged4_workspace_size
    assert size(1, 1, 1, 1, 16, 16, 1) == 0          # too little work for a second run
    assert size(32, 32, 16, 4, 128, 64, 128) > size(32, 32, 16, 4, 64, 64, 128) > 0
    for bad in ((0, 1, 8, 2), (1, 0, 8, 2), (1, 1, 7, 2), (1, 1, 0, 1), (1, 1, 8, 0)):
        assert size(*bad, 64, 16, 100) == 0
    assert size(1, 1, 8, 2, 48, 16, 100) == 0


def test_helpers_refuse_what_is_no_such_cache(lib):
    torch = pytest.importorskip("torch")
    sd._paged()
    pages = sd.paged4_pages(3, 2, 16, 64, device="cpu")
    assert pages.shape == (3, 2, 16, 36) and pages.dtype == torch.uint8
    i = torch.zeros(2, dtype=torch.int32)
    q, k = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens = i.view(1, 2), i[:1]
    # (tensors of the CPU: the device is what is refused)
    for call in (lambda: sd.paged4_attention(q, pages, pages.clone(), table, i, lens),
                 lambda: sd.paged4_append(q, k, k, pages, pages.clone(), table, i, lens),
                 lambda: sd.paged4_read(pages, pages, table, i, lens, k, k.clone())):
        with pytest.raises(sd.SdpaError) as e:
            call()
        assert e.value.status == INVALID
    with pytest.raises(TypeError):
        sd.paged4_attention(q, pages, None, table, i, lens)
    with pytest.raises(TypeError):
        sd.paged4_attention(q, pages, pages, table, i, lens, k_exp=0.5)
    with pytest.raises(OverflowError):
        sd.paged4_attention(q, pages, pages, table, i, lens, window=1 << 40)
    with pytest.raises(sd.SdpaError):
        sd.paged4_pages(1, 1, 16, 40)


def test_reference_quantises_to_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((300, 32)) * np.exp(3 * rng.standard_normal((300, 1)))
    for exp in (0, -4, 3):
        codes, scales = p4.quantise(x, exp)
        v = p4.values(codes, scales, exp)
        b = x.reshape(300, 2, 16)
        s = np.repeat(p4.E4M3[scales], 16, -1) * 2.0 ** exp
        grid = np.concatenate((-p4.GRID, p4.GRID))[None, None] * s[..., None]
        assert np.allclose(np.abs(x - v), np.abs(x[..., None] - grid).min(-1), atol=0)
        want = np.abs(b).max(-1) / 6 / 2.0 ** exp
        assert np.allclose(np.abs(p4.E4M3[scales] - want), np.abs(p4.E4M3 - want[..., None]).min(-1), atol=0)
    # ties go to the even code and the even scale
    one = np.zeros((1, 16))
    one[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    codes, scales = p4.quantise(one)
    assert p4.E4M3[scales[0, 0]] == 1.0 and list(codes[0, :8]) == [7, 0, 2, 2, 4, 4, 6, 6]
    one[0, :8] = 6 * (1 + 1 / 16)
    assert p4.E4M3[p4.quantise(one)[1][0, 0]] == 1.0
    one[0, :8] = 6 * (1 + 3 / 16)
    assert p4.E4M3[p4.quantise(one)[1][0, 0]] == 1.25
