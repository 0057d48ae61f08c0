"""Checks of the attention binding that need no GPU: CPU tensors stand in for GPU
ones, whose device number the checks compare (-1 for the CPU)."""
import types

import pytest
import torch

from group_dft_structured_amd import AttnPlan, EqlinearError, Packing

GO = types.SimpleNamespace(torch=torch, device=-1)


def _offsets(*values):
    return torch.tensor(values, dtype=torch.int32)


def test_packing_fields():
    cu = _offsets(0, 3, 7)
    f = Packing(cu, 4).fields(7, 7, GO)
    assert f[:5] == (2, 7, 7, 4, 4) and f[5] == f[6] == cu.data_ptr() and f[7:] == (0, 0)
    assert Packing(_offsets(0), 0).fields(0, 0, GO)[0] == 0


@pytest.mark.parametrize("shape", [(1, 3), (3, 1), (3, 2), (), (0,)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_packing_refuses_offsets_that_are_not_a_row(shape, which):
    # [1, B + 1] read as no sequence at all, [B + 1, 2] as every other offset
    bad = torch.zeros(shape, dtype=torch.int32)
    for cu in ((bad, None) if which == "q" else (_offsets(0, 3, 7), bad),
               (bad, bad) if which == "q" else (_offsets(0, 3, 7), bad)):
        with pytest.raises(ValueError):
            Packing(cu[0], 4, cu[1], 4).fields(7, 7, GO)


def test_packing_refuses_other_lengths_and_types():
    cu = _offsets(0, 3, 7)
    for bad in (_offsets(0, 7), cu.long(), torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            Packing(cu, 4, bad, 4).fields(7, 7, GO)
    with pytest.raises(ValueError):
        Packing(cu, 4, pos_q=torch.zeros(6, dtype=torch.int32)).fields(7, 7, GO)


def test_no_key_value_heads_are_refused():
    with pytest.raises(EqlinearError, match="EQL_ERR_INVALID_ARG"):
        AttnPlan(4, 64, kv_heads=0)
    plan = AttnPlan(4, 64)
    assert plan.Hk == 4


@pytest.mark.parametrize("scale", [1e39, 1e300])
def test_scales_beyond_binary32_are_refused(scale):
    # they would be an infinity in every score
    with pytest.raises(EqlinearError, match="EQL_ERR_INVALID_ARG"):
        AttnPlan(4, 64, scale=scale)
    AttnPlan(4, 64, scale=3e38)
