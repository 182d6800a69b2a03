"""Host tests of the layer norm and its backward: the oracle's pins, the C ABI's
refusals (fake device addresses; every call returns before a HIP call) and the
binding's argument checks. No GPU needed, no kernel is launched."""
import numpy as np
import pytest
import torch

import invariant_token_log_fp32_amd as rlk
from oracle import layer_norm as LN

OK, NULL, ALIGN, SHAPE, WS = 0, -1, -2, -3, -5
P = 0x10000
META = torch.device("meta")


@pytest.mark.parametrize("rms", [False, True])
def test_oracle_against_torch_autograd(rms):
    rng = np.random.default_rng(0)
    x = torch.tensor(rng.normal(1, 2, (6, 40)), requires_grad=True)
    w = torch.tensor(rng.normal(1, 1, 40), requires_grad=True)
    b = torch.tensor(rng.normal(0, 1, 40), requires_grad=True)
    dy = torch.tensor(rng.normal(0, 1, (6, 40)))
    if rms:
        y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-3) * w + b
    else:
        y = torch.nn.functional.layer_norm(x, (40,), w, b, 1e-3)
    y.backward(dy)
    got, m, r = LN.forward(x.detach().numpy(), w.detach().numpy(), b.detach().numpy(), 1e-3, rms)
    assert np.allclose(got, y.detach().numpy(), atol=1e-12)
    dx, dw, db = LN.backward(dy.numpy(), x.detach().numpy(), w.detach().numpy(), m, r, rms)
    for a, t in ((dx, x), (dw, w), (db, b)):
        assert np.allclose(a, t.grad.numpy(), atol=1e-12)


def test_every_declared_function_is_exported():
    names = rlk.declared_functions(rlk.TRAINING_HEADER_PATHS)
    assert {"rlk_layer_norm", "rlk_layer_norm_backward", "rlk_layer_norm_backward_workspace_bytes"} <= set(names)
    for n in names:
        assert getattr(rlk.load_library(), n).argtypes is not None, n


def test_workspace_sizes():
    f = rlk.layer_norm_backward_workspace_bytes
    assert f(8192, 4096) >= 2 * 4 * 4096
    for n, d in ((-1, 64), ((1 << 22) + 1, 64), (1, 0), (1, 4), (1, 60), (1, 16392)):
        assert f(n, d) == 0, (n, d)
    for d in (8, 1000, 4096, 16384):
        last = 0
        for n in (0, 1, 5, 100, 1000, 5000, 100000):
            assert f(n, d) >= last
            last = f(n, d)


def fwd(x=P, xt=0, n=4, d=64, ldx=64, w=2 * P, b=3 * P, wt=0, kind=0, eps=1e-6, y=4 * P, ldy=64, mean=5 * P, rstd=6 * P):
    return rlk.load_library().rlk_layer_norm(x, xt, n, d, ldx, w, b, wt, kind, eps, y, ldy, mean, rstd, None)


SIZES = [(dict(n=-1), SHAPE), (dict(n=(1 << 22) + 1), SHAPE), (dict(d=0), SHAPE), (dict(d=60), SHAPE), (dict(d=16392, ldx=16392), SHAPE),
         (dict(ldx=56), SHAPE), (dict(ldx=68), SHAPE), (dict(ldx=1 << 40), SHAPE), (dict(xt=2), SHAPE), (dict(xt=-1), SHAPE),
         (dict(wt=2), SHAPE), (dict(kind=2), SHAPE)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(ldy=56), SHAPE), (dict(ldy=65), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(x=P + 8), ALIGN), (dict(w=P + 8), ALIGN), (dict(b=P + 8), ALIGN), (dict(y=P + 8), ALIGN), (dict(mean=P + 2), ALIGN),
    (dict(rstd=P + 2), ALIGN), (dict(n=0, x=None, w=None, y=None), OK),
    (dict(y=P, ldy=128), SHAPE), (dict(y=P, ldx=128), SHAPE), (dict(y=P, xt=1), SHAPE),
])
def test_forward_refuses(kw, code):
    assert fwd(**kw) == code


def bwd(dy=P, lddy=64, x=2 * P, xt=0, n=4, d=64, ldx=64, w=3 * P, wt=0, kind=0, mean=4 * P, rstd=5 * P, dx=6 * P, lddx=64, dw=7 * P,
        db=8 * P, acc=0, ws=9 * P, wb=1 << 30):
    return rlk.load_library().rlk_layer_norm_backward(dy, lddy, x, xt, n, d, ldx, w, wt, kind, mean, rstd, dx, lddx, dw, db, acc, ws, wb,
                                                      None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dx=2 * P, lddx=128), SHAPE), (dict(dx=P, lddx=128), SHAPE), (dict(dx=P, xt=1), SHAPE), (dict(dx=2 * P, ldx=128), SHAPE),
    (dict(lddy=56), SHAPE), (dict(lddy=66), SHAPE), (dict(lddx=56), SHAPE), (dict(lddx=66), SHAPE), (dict(acc=2), SHAPE),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL),
    (dict(dx=None, dw=None, db=None), NULL), (dict(ws=None), NULL),
    (dict(dy=P + 8), ALIGN), (dict(x=P + 8), ALIGN), (dict(w=P + 8), ALIGN), (dict(mean=P + 2), ALIGN), (dict(rstd=P + 2), ALIGN),
    (dict(dx=P + 8), ALIGN), (dict(dw=P + 8), ALIGN), (dict(db=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(wb=100), WS),
    (dict(n=0, dw=None, db=None), OK), (dict(n=0, acc=1), OK),
])
def test_backward_refuses(kw, code):
    assert bwd(**kw) == code


def test_binding_checks_tensors():
    x = torch.empty((4, 64), dtype=torch.bfloat16, device=META)
    w = torch.empty(64, dtype=torch.bfloat16, device=META)
    assert rlk._matrix(x, "x") == (64, rlk.TYPE_BF16)
    assert rlk._matrix(x[:1], "x") == (64, rlk.TYPE_BF16)
    assert rlk._norm_weight(w, None, 64, META) == rlk.TYPE_BF16
    for bad in (torch.zeros((4, 64), dtype=torch.bfloat16), x.to(torch.float16), x[0], x[:, ::2], None, x[None]):
        with pytest.raises(ValueError):
            rlk._matrix(bad, "x")
    with pytest.raises(ValueError):
        rlk._matrix(x.float(), "out", f32_too=False)
    with pytest.raises(ValueError, match="of shape"):
        rlk._matrix(x[:3], "grad_x", x)
    for weight, bias in ((None, None), (w.to(torch.float16), None), (w[:32], None), (w, w.float()), (torch.zeros(64), None)):
        with pytest.raises(ValueError):
            rlk._norm_weight(weight, bias, 64, META)
    with pytest.raises(ValueError, match="accumulate"):
        rlk.layer_norm_backward(x, x, w, torch.empty(4, device=META), torch.empty(4, device=META), accumulate=True)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=META)
    with pytest.raises(ValueError, match="x on meta"):
        rlk.layer_norm(x, None, stream=Stream())
    with pytest.raises(ValueError, match="grad_out on meta"):
        rlk.layer_norm_backward(x, x, None, None, None, stream=Stream())
