"""Serving calls without a token, on tensors whose strides say nothing: an array
without elements has strides of zero, and so has the tensor made of it."""
import numpy as np
import pytest

import transformer_scaled_dot_02_gb300 as sd
from gpu_util import dev, dev_int

pytestmark = pytest.mark.gpu


def _rows(heads, d):
    import torch
    x = torch.from_numpy(np.zeros((0, heads, d), np.float32)).bfloat16().cuda()
    return x.as_strided((0, heads, d), (0, 0, 0))


@pytest.mark.parametrize("held", ["bf16", "4 bits"])
def test_calls_without_a_token(held):
    import torch
    h, h_kv, d, page, b = 4, 2, 64, 16, 3
    table = dev_int(np.arange(6).reshape(b, 2))
    starts, lens = dev_int([0] * (b + 1)), dev_int([20, 0, 32])
    q, k, v = _rows(h, d), _rows(h_kv, d), _rows(h_kv, d)
    assert q.stride(2) == 0
    if held == "bf16":
        pages = [torch.ones(6, h_kv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        append, attention = sd.paged_append, sd.paged_attention
    else:
        pages = [torch.full((6, h_kv, page, 9 * d // 16), 17, dtype=torch.uint8, device="cuda") for _ in range(2)]
        append, attention = sd.paged4_append, sd.paged4_attention
        got = sd.paged4_read(*pages, table, starts, lens, k, v)
        assert got[0] is k and got[1] is v
    before = [x.clone() for x in pages]
    assert append(q, k, v, *pages, table, starts, lens).shape == (0, h, d)
    assert append(None, k, v, *pages, table, starts, lens) is None
    assert attention(q, *pages, table, starts, lens).shape == (0, h, d)
    out = _rows(h, d)
    assert attention(q, *pages, table, starts, lens, out=out) is out
    assert all(torch.equal(x, y) for x, y in zip(pages, before))
    sd.sdpa_device_check()


def test_what_is_no_empty_tensor_of_these_shapes_is_refused():
    h_kv, d = 2, 64
    pages = [sd.paged4_pages(6, h_kv, 16, d) for _ in range(2)]
    rest = (dev_int(np.arange(6).reshape(3, 2)), dev_int([0] * 4), dev_int([20, 0, 32]))
    for q in (_rows(4, 32), dev(np.zeros((0, 4, d), np.float32), "f32"), dev(np.zeros((2, 4, d), np.float32))[:, :, ::2]):
        with pytest.raises(sd.SdpaError):
            sd.paged4_attention(q, *pages, *rest)
