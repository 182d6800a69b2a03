"""The last position of one sequence, hidden[:, -1] of a [1, length, d] tensor, through every
entry point that takes hidden states: a matrix of one row whose stride (length * d, beyond
what several rows may have) has no meaning. The bytes are those of a copy of the row."""
import pytest

import invariant_token_log_fp32_amd as rlk

from gpu_util import say

pytestmark = pytest.mark.gpu

D, LENGTH, VR, VP = 256, 8193, 1000, 1024


def last(dtype, seed=0, length=LENGTH):
    """A [1, D] view, the last row of a sequence whose other rows hold NaN, and a copy of it."""
    import torch
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    buf = torch.full((1, length, D), float("nan"), dtype=dtype, device="cuda:0")
    buf[:, -1] = torch.randn((1, D), generator=gen, device="cuda:0").to(dtype)
    view = buf[:, -1]
    assert view.stride(0) == length * D > 1 << 21
    return view, view.contiguous().clone()


def weights(dtype):
    import torch
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    return (torch.randn((VR, D), generator=gen, device="cuda:0") / 8).to(dtype), torch.rand(D, generator=gen, device="cuda:0").to(dtype)


@pytest.mark.parametrize("length", [LENGTH, LENGTH + 1])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_norm(dtype, length):
    import torch
    say(f"case: norm of the last of {length} positions, {dtype}")
    x, copy = last(getattr(torch, dtype), length=length)
    _, gain = weights(torch.float32)
    dy, dy_copy = last(torch.bfloat16, 2)
    out = last(torch.bfloat16, 3)[0]
    want = rlk.layer_norm(copy, gain, return_stats=True)
    for got in (rlk.layer_norm(x, gain, return_stats=True), rlk.layer_norm(x, gain, return_stats=True, out=out)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    want_g = rlk.layer_norm_backward(dy_copy, copy, gain, *want[1:], bias_grad=True)
    grad_x = last(getattr(torch, dtype), 4)[0]
    for kw in (dict(), dict(grad_x=grad_x)):
        got = rlk.layer_norm_backward(dy, x, gain, *want[1:], bias_grad=True, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want_g))
    got = rlk.layer_norm_backward(dy, x, gain, *want[1:], grad_x=x)  # in place
    assert got[0] is x and torch.equal(x, want_g[0])


def test_head():
    import torch
    say("case: the head on the last position")
    x, copy = last(torch.bfloat16)
    w, _ = weights(torch.bfloat16)
    t, tg = torch.ones(1, device="cuda:0"), torch.full((1,), 7, dtype=torch.int64, device="cuda:0")
    assert torch.equal(rlk.linear(x, w, vocab_padded=VP), rlk.linear(copy, w, vocab_padded=VP))
    logp, lse = rlk.linear_logp(copy, w, t, tg, vocab_padded=VP, return_lse=True)
    assert torch.equal(rlk.linear_logp(x, w, t, tg, vocab_padded=VP), logp)
    kw = dict(vocab_padded=VP, ref_logp=logp, lse=lse, grad_ref=torch.ones_like(logp))
    want = rlk.linear_logp_backward(copy, w, t, tg, **kw)
    out = last(torch.bfloat16, 5)[0]
    for more in (dict(), dict(grad_hidden=out)):
        got = rlk.linear_logp_backward(x, w, t, tg, **kw, **more)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    parts = rlk.linear_logp_backward(copy, w, t, tg, **kw, grad_hidden=torch.empty((1, D), device="cuda:0"))[0]
    merged = rlk.linear_logp_backward_merge(parts[None], out=last(torch.bfloat16, 6)[0])
    assert torch.equal(merged, want[0])
    a, b = rlk.mx4_quantize(x, return_values=True), rlk.mx4_quantize(copy, return_values=True)
    assert torch.equal(a[2], b[2])
