"""mdl_distill where its range or its rules end: weight 0 beside classes that do not exist, temperatures whose square is
no fp32 number, rows longer than the registers hold, and rows near 2^31 classes. Tolerances are test_gpu_distill.py's."""

import numpy as np
import pytest
import torch

from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from test_gpu_distill import DEV, check, make, run


@pytest.mark.parametrize("V,dtype", [(7, "f32"), (300, "bf16"), (5003, "f32")])
def test_weight_zero_wins_over_a_class_that_does_not_exist(V, dtype):
    """A padded frame whose ids were never set: loss 0 and gradient 0, like any other of weight 0."""
    z, ids, t, w = make(21, 6, V, 4, dtype)
    ids[1], w[1] = V, 0.0
    ids[2, 0], ids[2, 1], w[2] = -1, -5, 0.0
    ids[3, 2] = V + 1                               # with a weight: NaN
    ids[4], w[4], z[4], t[4] = 2 ** 31 - 1, 0.0, float("nan"), float("nan")
    _, loss, dz = run(z, ids, t, w, 1.5, dtype)
    assert not loss[[1, 2, 4]].any() and torch.isnan(loss[3]) and not dz[1:5].any()
    assert torch.isfinite(loss[[0, 5]]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1e-30, 1e-25, 1e-20, 3e-19, 1e15, 1e17])
def test_temperatures_whose_square_is_no_fp32_number(tau, dtype):
    """Sharp ones: the loss is w tau times the difference of the largest logits' gaps. Flat ones keep few classes, so
    that the loss, about w tau^2 ln(V / k), is within fp32."""
    z, ids, t, w = make(22, 9, 900, 6, dtype)
    _, loss, _ = run(z, ids, t, w, tau, dtype)
    assert torch.isfinite(loss).all() and (loss > 0).any()
