"""The paged entry points on the CPU: argument checks return their documented
codes, the workspace size follows the shapes, and the fp64 reference that the
GPU tests use agrees with the oracle and with the rotation's own laws."""
import ctypes

import numpy as np
import pytest

import oracle
import paged_util as pu
import synthetic
import transformer_scaled_dot_02_gb300 as sd
from transformer_scaled_dot_02_gb300 import build as sd_build

INVALID, UNSUPPORTED, NODEV, WORKSPACE = 1, 2, 3, 4
A, MIS = 0x10000, 0x10008       # placeholder addresses: no call below reaches CUDA work


def _gpu_visible():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


@pytest.fixture(scope="module")
def lib():
    sd_build.build()
    oracle.build()
    return sd.load_library()


SHAPE = dict(b=3, t=5, h=8, h_kv=2, d=64, page=16, n_pages=40, per_seq=12, table=A, starts=A, lens=A)


def _append(lib, **kw):
    a = dict(SHAPE, q=A, k=A, v=A, q_out=2 * A, kp=A, vp=A, qs=512, ks=128, vs=128, freqs=A, d_rot=64, inter=0)
    a.update(kw)
    return lib.sdpa_paged_append(a["q"], a["k"], a["v"], a["q_out"], a["kp"], a["vp"], a["b"], a["t"], a["h"],
                                 a["h_kv"], a["d"], a["page"], a["n_pages"], a["per_seq"], a["table"],
                                 a["starts"], a["lens"], a["qs"], a["ks"], a["vs"], a["freqs"], a["d_rot"],
                                 a["inter"], None)


def _forward(lib, **kw):
    a = dict(SHAPE, q=A, kp=A, vp=A, out=2 * A, ws=A, ws_bytes=1 << 40, qs=512, scale=0.0)
    a.update(kw)
    return lib.sdpa_paged_forward(a["q"], a["kp"], a["vp"], a["out"], a["ws"], a["ws_bytes"], a["b"], a["t"],
                                  a["h"], a["h_kv"], a["d"], a["page"], a["n_pages"], a["per_seq"], a["table"],
                                  a["starts"], a["lens"], a["qs"], ctypes.c_float(a["scale"]), None)


@pytest.mark.parametrize("call", [_append, _forward])
def test_shared_argument_checks(lib, call):
    for name in ("kp", "vp", "table", "starts", "lens"):
        assert call(lib, **{name: None}) == INVALID, name
    assert call(lib, kp=MIS) == INVALID
    assert call(lib, vp=MIS) == INVALID
    for name in ("table", "starts", "lens"):
        assert call(lib, **{name: A + 2}) == INVALID, name
    for name, value in (("b", 0), ("t", -1), ("h", 0), ("h_kv", 0), ("d", 0), ("page", 0), ("n_pages", 0),
                        ("per_seq", 0), ("h_kv", 3)):
        assert call(lib, **{name: value}) == INVALID, (name, value)
    for d in (8, 48, 96, 512):
        assert call(lib, d=d, h=2, h_kv=2, qs=4096) == UNSUPPORTED, d
    for page in (1, 4, 24, 100):
        assert call(lib, page=page) == UNSUPPORTED, page
    assert call(lib, h=129, h_kv=1, qs=129 * 64) == UNSUPPORTED
    assert call(lib, per_seq=1 << 26) == UNSUPPORTED          # 2^30 positions
    assert call(lib, t=(1 << 24) + 1) == UNSUPPORTED
    assert call(lib, h=64, h_kv=64, d=16, qs=1024, page=1 << 25, per_seq=1, n_pages=1) == UNSUPPORTED
    assert call(lib, n_pages=1 << 30) == UNSUPPORTED


def test_append_argument_checks(lib):
    for name in ("k", "v"):
        assert _append(lib, **{name: None}) == INVALID
    assert _append(lib, q=None) == INVALID                    # q_out without q, and the reverse
    assert _append(lib, q_out=None) == INVALID
    for name in ("q", "k", "v", "q_out"):
        assert _append(lib, **{name: MIS}) == INVALID, name
    assert _append(lib, qs=511) == INVALID
    assert _append(lib, ks=120) == INVALID
    assert _append(lib, vs=0) == INVALID
    assert _append(lib, qs=516) == UNSUPPORTED                # rows must start on 16 bytes
    assert _append(lib, ks=132) == UNSUPPORTED
    assert _append(lib, vs=129) == UNSUPPORTED
    assert _append(lib, d_rot=-16) == INVALID
    assert _append(lib, d_rot=80) == INVALID
    assert _append(lib, d_rot=24) == UNSUPPORTED
    assert _append(lib, freqs=None) == INVALID
    assert _append(lib, freqs=A + 2) == INVALID
    # in place only where the rows are dense
    assert _append(lib, q=A, q_out=A, qs=768) == INVALID
    # rotated queries on the rows of another operand, or partly on their own
    far = 16 * A
    assert _append(lib, q=far, k=A, v=far, q_out=A) == INVALID
    assert _append(lib, q=far, k=far, v=A, q_out=A + 64) == INVALID
    assert _append(lib, q=A, k=far, v=far, q_out=A + 1024) == INVALID
    if not _gpu_visible():
        assert _append(lib, q=A, k=far, v=far, q_out=A, qs=512) == NODEV
        assert _append(lib, q=A, k=far, v=far, q_out=A + 5 * 1024, qs=512) == NODEV
        assert _forward(lib, out=A + 5 * 1024) == NODEV


def test_forward_argument_checks(lib):
    assert _forward(lib, q=None) == INVALID
    assert _forward(lib, out=None) == INVALID
    assert _forward(lib, q=MIS) == INVALID
    assert _forward(lib, out=MIS) == INVALID
    assert _forward(lib, qs=504) == INVALID
    assert _forward(lib, qs=516) == UNSUPPORTED
    # the output must not lie on the queries: 5 rows of 1024 bytes
    for out in (A, A + 1024, A + 4 * 1024, A - 16, A - 4 * 1024):
        assert _forward(lib, out=out) == INVALID, out
    assert _forward(lib, out=A + 5 * 1024, scale=-1.0) == INVALID
    for scale in (-1.0, float("nan"), float("inf")):
        assert _forward(lib, scale=scale) == INVALID
    need = sd.sdpa_paged_workspace_size(3, 5, 8, 2, 64, 16, 12)
    assert need > 0
    assert _forward(lib, ws=None) == WORKSPACE
    assert _forward(lib, ws=MIS) == WORKSPACE
    assert _forward(lib, ws_bytes=need - 1) == WORKSPACE


@pytest.mark.skipif(_gpu_visible(), reason="valid placeholder arguments would reach a real GPU")
def test_valid_arguments_without_gpu_report_no_device(lib):
    assert _append(lib) == NODEV
    assert _append(lib, q=None, q_out=None) == NODEV
    assert _append(lib, qs=768, ks=768, vs=768, freqs=None, d_rot=0) == NODEV
    assert _forward(lib) == NODEV
    assert _forward(lib, t=0, q=None, out=None, ws=None, ws_bytes=0) == NODEV
    assert _append(lib, t=0, q=None, k=None, v=None, q_out=None) == NODEV


def test_workspace_size_follows_the_shapes(lib):
    size = sd.sdpa_paged_workspace_size
    assert size(0, 1, 1, 1, 64, 16, 4) == 0
    assert size(1, 0, 1, 1, 64, 16, 4) == 0
    assert size(1, 1, 3, 2, 64, 16, 4) == 0
    assert size(1, 1, 1, 1, 96, 16, 4) == 0
    assert size(1, 1, 1, 1, 64, 16, 3) == 0                   # one run: nothing to merge
    small, large = size(1, 1, 8, 8, 64, 16, 64), size(64, 4096, 8, 8, 64, 16, 64)
    assert 0 < small < large
    # never more than four slots of 128 rows for every three resident CTAs
    assert size(1 << 12, 1 << 20, 16, 16, 128, 64, 2048) <= 4 * 2 * 152 * 128 * 130 * 4 // 3 + (1 << 18)
    # ... and bounded by the rows of the call
    assert size(1, 1, 8, 1, 128, 64, 2048) <= 4 * 2 * 152 * 8 * 130 * 4 // 3 + (1 << 18)


def _cpu_tensors(torch):
    rows = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, ints = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    return rows, pages, table, ints


def test_helpers_refuse_what_the_library_cannot_see(lib):
    """Tensors on the CPU are refused before the library is asked."""
    torch = pytest.importorskip("torch")
    rows, pages, table, ints = _cpu_tensors(torch)
    with pytest.raises(sd.SdpaError):
        sd.paged_attention(rows, pages, pages, table, ints, ints[:1], workspace=ints)
    with pytest.raises(sd.SdpaError):
        sd.paged_append(rows, rows, rows, pages, pages, table, ints, ints[:1])
    with pytest.raises(sd.SdpaError):
        sd.paged_append(None, rows, rows, pages, pages, table, ints, ints[:1])


def test_helpers_refuse_what_is_no_tensor(lib):
    torch = pytest.importorskip("torch")
    rows, pages, table, ints = _cpu_tensors(torch)
    for at in range(1, 6):
        args = [rows, pages, pages, table, ints, ints[:1]]
        args[at] = None if at != 3 else 7
        with pytest.raises((TypeError, AttributeError)):
            sd.paged_attention(*args, workspace=ints)
    for at in range(1, 8):
        args = [rows, rows, rows, pages, pages, table, ints, ints[:1]]
        args[at] = None if at != 3 else A
        with pytest.raises(TypeError):
            sd.paged_append(*args)
    with pytest.raises(TypeError):
        sd.paged_attention(rows, pages, pages, table, ints, ints[:1], scale="1", workspace=ints)


def _bf16(rng, shape):
    return synthetic.round_to_bf16(rng.standard_normal(shape).astype(np.float32))


def test_reference_is_the_oracles_decoding_step(lib):
    """One kv head per query head, n_q new tokens each: the paged reference
    and the oracle's decode are the same function."""
    rng = np.random.default_rng(1)
    b, h, n_q, n_k, d = 3, 2, 3, 50, 16
    k, v, q = _bf16(rng, (b, h, n_k, d)), _bf16(rng, (b, h, n_k, d)), _bf16(rng, (b, h, n_q, d))
    lens = np.array([50, 2, 17], np.int32)
    ref = oracle.decode(q, k, v, lens)
    packed = q.transpose(0, 2, 1, 3).reshape(b * n_q, h, d)
    dense = [[x[s, :, :lens[s]].transpose(1, 0, 2) for s in range(b)] for x in (k, v)]
    out, bound = pu.attention(packed, *dense, pu.starts_of([n_q] * b), lens)
    got = out.reshape(b, n_q, h, d).transpose(0, 2, 1, 3)
    assert np.abs(got - ref).max() <= 1e-6          # the oracle returns fp32
    assert np.all(bound >= 0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32)), pu.freqs_of(32)
    at = lambda x, p: pu.rotate(x, np.array([p]), f, interleaved)[0].ravel()
    assert np.isclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q))
    assert np.isclose(at(q, 1007) @ at(k, 1000), at(q, 7) @ at(k, 0))
    assert np.array_equal(at(q, 0), q.ravel())
