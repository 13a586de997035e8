"""IF4 planes have NVFP4's shapes and other values in their blocks of integers: they make no weight."""
import copy
import pickle

import pytest
import torch

import fp4_block_scaled_row_amd as fq


def made(policy):
    planes = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), torch.ones(1)
    r = fq.NvResult(*planes, None, None, None)
    r.policy = policy
    return r


@pytest.mark.parametrize("again", [lambda r: r, copy.copy, lambda r: r._replace(rotated=None),
                                   lambda r: pickle.loads(pickle.dumps(r))])
def test_if4_results_are_refused(again):
    with pytest.raises(ValueError, match="IF4"):
        fq.fp4_weight(again(made("if4")))
    for policy in (None, "max6", "four_over_six"):
        with pytest.raises(ValueError, match="GPU"):        # (as far as planes on the CPU go)
            fq.fp4_weight(again(made(policy)))


def test_results_are_the_tuples_they_were():
    r = made("max6")
    codes, scales, g, choice, rotated, counters = r
    assert isinstance(r, tuple) and len(r) == 6 and r[0] is codes is r.codes and r[2] is g
    assert r._fields == ("codes", "scales", "global_scale", "choice_bits", "rotated", "counters")
    assert fq.NvResult(codes, scales, g, choice, rotated, counters).policy is None


@pytest.mark.gpu
def test_the_last_policy_counts():
    x = torch.randn(8, 64, device="cuda")
    q = fq.quantize_nvfp4(x, policy="if4")
    with pytest.raises(ValueError, match="IF4"):
        fq.fp4_weight(q)
    assert fq.quantize_nvfp4(x, out=q) is q and fq.fp4_weight(q).format == "nvfp4"
    fq.quantize_nvfp4(x, policy="if4", out=q)
    with pytest.raises(ValueError, match="IF4"):
        fq.fp4_weight(q)
    for policy in ("max6", "four_over_six"):
        assert fq.fp4_weight(fq.quantize_nvfp4(x, policy=policy)).n == 8
