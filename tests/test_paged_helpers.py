"""What the paged helpers answer to tensors that do not fit: the library's
status, whether a workspace is given or not."""
import numpy as np
import pytest

import paged_util as pu
import transformer_scaled_dot_02_gb300 as sd
from transformer_scaled_dot_02_gb300 import build as sd_build
from gpu_util import host

torch = pytest.importorskip("torch")


def _tensors(device):
    rows = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=device)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=device)
    table, ints = (torch.zeros(s, dtype=torch.int32, device=device) for s in ((1, 2), (2,)))
    return [rows, pages, pages, table, ints, ints[:1]]


def _unfit(args):
    """Each of them with a tensor of another rank in one place."""
    rows, pages, _, table, ints, _ = args
    for at, x in ((0, rows[0]), (0, rows[None]), (1, pages[0]), (1, pages[None]), (2, pages[0]), (3, table[0]),
                  (3, table[None]), (4, table), (5, table)):
        bad = list(args)
        bad[at] = x
        yield bad


def _check_refusals(device):
    args = _tensors(device)
    for given in ({}, {"workspace": torch.empty(1 << 20, dtype=torch.uint8, device=device)}):
        for bad in _unfit(args):
            with pytest.raises(sd.SdpaError) as e:
                sd.paged_attention(*bad, **given)
            assert e.value.status == 1
        for at in range(6):
            for x in (None, 7):
                bad = list(args)
                bad[at] = x
                with pytest.raises(TypeError):
                    sd.paged_attention(*bad, **given)


def test_refusals_do_not_depend_on_the_workspace():
    sd_build.build()
    _check_refusals("cpu")


@pytest.mark.gpu
def test_refusals_do_not_depend_on_the_workspace_on_the_gpu():
    _check_refusals("cuda")
    sd.sdpa_device_check()


@pytest.mark.gpu
def test_a_workspace_is_made_where_one_is_needed():
    """One run needs none, several do; the same result as with one that is given."""
    for n_pages, per_seq in ((4, 2), (130, 128)):
        rng = torch.Generator("cuda").manual_seed(n_pages)
        normal = lambda *s: torch.randn(*s, generator=rng, dtype=torch.bfloat16, device="cuda")
        q, kp, vp = normal(1, 8, 64), normal(n_pages, 2, 16, 64), normal(n_pages, 2, 16, 64)
        table = torch.arange(per_seq, dtype=torch.int32, device="cuda")[None]
        starts, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [16 * per_seq]))
        ws = sd.paged_workspace(q, kp, table)
        args = (q, kp, vp, table, starts, lens)
        assert torch.equal(sd.paged_attention(*args), sd.paged_attention(*args, workspace=ws))
        dense = [[host(x[table[0].long()].transpose(1, 2).flatten(0, 1))] for x in (kp, vp)]
        want, bound = pu.attention(host(q), *dense, [0, 1], [16 * per_seq])
        assert np.all(np.abs(host(sd.paged_attention(*args)) - want) <= bound)
    sd.sdpa_device_check()


@pytest.mark.gpu
def test_keys_and_values_in_one_place_are_refused_by_the_append_alone():
    rows, pages, _, table, ints, lens = _tensors("cuda")
    starts, lens = ints + torch.tensor([0, 1], dtype=torch.int32, device="cuda"), lens + 5
    both = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    for kp, vp in ((pages, pages), (both[:4], both[1:]), (both[1:], both[:4])):
        with pytest.raises(sd.SdpaError) as e:
            sd.paged_append(rows, rows, rows, kp, vp, table, starts, lens)
        assert e.value.status == 1
        assert torch.all(sd.paged_attention(rows, kp, vp, table, starts, lens) == 0)
    kp, vp = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")     # side by side is well
    sd.paged_append(rows, rows + 1, rows + 2, kp, vp, table, starts, lens)
    assert kp[0, :, 4].eq(1).all() and vp[0, :, 4].eq(2).all()
    assert kp.sum() == 128 and vp.sum() == 256
    sd.sdpa_device_check()
