"""The training head's workspaces at exactly the size that is asked for: what lies behind them
stays as it was, what they hold before the call (NaN patterns) does not matter, and a
workspace used by one call after another gives each its own result."""
import pytest

import invariant_token_log_fp32_amd as rlk

from gpu_util import say
from test_gpu_linear_grad import Problem

pytestmark = pytest.mark.gpu

BEHIND = 4096


def exact(need):
    """(workspace of `need` bytes, the bytes behind it), both 0xFF: NaN in every type."""
    import torch
    buf = torch.full((need + BEHIND,), 0xFF, dtype=torch.uint8, device="cuda:0")
    return buf[:need], buf[need:]


HEADS = [(1, 64, 1, 64), (1, 128, 300, 320), (63, 64, 5000, 5056), (129, 192, 2111, 2176), (257, 320, 1000, 1024), (515, 576, 3001, 8192),
         (1025, 64, 500, 512), (3000, 64, 40000, 40064), (4096, 4096, 500, 512)]


@pytest.mark.parametrize("n,d,vr,vp", HEADS)
def test_gradient_of_the_head(n, d, vr, vp):
    import torch
    say(f"case: {n} x {d} x {vr} of {vp}")
    p = Problem(n, n, d, vr, vp)
    a, kw = p.args()
    want = rlk.linear_logp_backward(*a, **kw)
    ws, behind = exact(rlk.linear_logp_backward_workspace_bytes(n, d, vp, vr))
    for up in (kw["grad_ref"].clone(), torch.where(torch.arange(n, device="cuda:0") % 3 == 0, kw["grad_ref"], 0.0), kw["grad_ref"].clone()):
        got = rlk.linear_logp_backward(*a, **dict(kw, grad_ref=up), workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((behind == 0xFF).all())
    for groups in (2, 8):
        cols = vp // groups
        parts = torch.empty((groups, n, d), device="cuda:0")
        for rank in range(groups):
            ws, behind = exact(rlk.linear_logp_backward_workspace_bytes(n, d, vp, vr, groups))
            w = p.w[min(vr, rank * cols):min(vr, (rank + 1) * cols)]
            rlk.linear_logp_backward(a[0], w, *a[2:], **kw, vocab_real=vr, rank=rank, groups=groups, grad_hidden=parts[rank], workspace=ws)
            assert bool((behind == 0xFF).all())
        assert torch.equal(rlk.linear_logp_backward_merge(parts), want[0])


@pytest.mark.parametrize("n,d", [(1, 8), (127, 1000), (128, 4096), (129, 8), (769, 4096), (1000, 16384), (4000, 1032), (40000, 1032), (70000, 64)])
@pytest.mark.parametrize("x32", [False, True])
def test_backward_of_the_norm(n, d, x32):
    import torch
    say(f"case: {n} x {d}, x32 {x32}")
    gen = torch.Generator(device="cuda:0").manual_seed(n)
    x = torch.randn((n, d), generator=gen, device="cuda:0")
    x = x if x32 else x.to(torch.bfloat16)
    dy = torch.randn((n, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    w = torch.rand(d, generator=gen, device="cuda:0") + 0.5
    _, mean, rstd = rlk.layer_norm(x, w, return_stats=True)
    want = rlk.layer_norm_backward(dy, x, w, mean, rstd, bias_grad=True)
    ws, behind = exact(rlk.layer_norm_backward_workspace_bytes(n, d))
    for _ in range(2):
        got = rlk.layer_norm_backward(dy, x, w, mean, rstd, bias_grad=True, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((behind == 0xFF).all())
    alone = x.clone()  # in place: the walk's sums for few rows too
    rlk.layer_norm_backward(dy, alone, w, mean, rstd, bias_grad=True, grad_x=alone, workspace=ws)
    assert torch.equal(alone, want[0]) and bool((behind == 0xFF).all())
