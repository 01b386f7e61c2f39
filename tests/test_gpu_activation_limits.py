"""Activations and their slopes at infinities and in the negative tails."""
import numpy as np
import pytest
import torch

from all_mxfp8_block_gb300 import mxa2a
from tests import operators_ref as R
from tests.test_gpu_linear import ACT
from tests.test_gpu_moe import TYPE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_slope_at_infinities(act):
    # the slopes' limits: 1 at +inf, 0 at -inf; a NaN stays one
    inf = float("inf")
    z = torch.tensor([inf, -inf, float("nan"), 3e38, -3e38] + [1.0] * 27).bfloat16().cuda()[None]
    one = torch.ones(1, 32, dtype=torch.bfloat16, device="cuda")
    l = mxa2a.Linear(1, 1, 32, 32, training=True)
    db = torch.full((1, 32), 7.0, device="cuda")
    l.backward(1, one, z, ACT[act], TYPE["e4m3"], None, None, None, None, None, None, 0, db)
    got = R.f64(db)[0]
    assert np.isnan(got[2])
    assert np.abs(got[[0, 1, 3, 4]] - [1, 0, 1, 0]).max() <= 1e-6, got[:5]
