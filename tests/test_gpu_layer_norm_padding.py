"""Rows of the norm's backward whose dy holds only zeros have dx = 0, whatever x, the
statistics and the weight hold: an infinity or NaN in the weight reaches the rows that have
a gradient, not the padding."""
import numpy as np
import pytest

import invariant_token_log_fp32_amd as rlk

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d", [(5, 72), (90, 1032), (300, 1032), (260, 4104), (140, 8200)])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_weight_that_is_no_number(n, d, rms, value):
    import torch
    say(f"case: {n} x {d}, rms {rms}, weight {value}")
    gen = torch.Generator(device="cuda:0").manual_seed(n)
    x = torch.randn((n, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    w = torch.rand(d, generator=gen, device="cuda:0") + 0.5
    dy = torch.randn((n, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    off = torch.rand(n, generator=gen, device="cuda:0") < 0.5
    off[0], off[1] = True, False
    dy[off] = 0
    dy[off, 3] = -0.0
    _, mean, rstd = rlk.layer_norm(x, w, return_stats=True)
    clean = rlk.layer_norm_backward(dy, x, w, mean, rstd, rms=rms, bias_grad=True)
    w[d - 5] = value
    dx, dw, db = rlk.layer_norm_backward(dy, x, w, mean, rstd, rms=rms, bias_grad=True)
    assert bool((dx[off] == 0).all())
    assert not dx[~off].isfinite().any()  # the sums over the row hold the weight
    assert torch.equal(dw, clean[1]) and torch.equal(db, clean[2])  # they do not hold the weight
    alone = dy.clone()
    rlk.layer_norm_backward(alone, x, w, mean, rstd, rms=rms, grad_x=alone)
    assert np.array_equal(alone.view(torch.int16).cpu().numpy() & 0x7FFF, dx.view(torch.int16).cpu().numpy() & 0x7FFF)
