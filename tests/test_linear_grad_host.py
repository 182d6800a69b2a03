"""Host tests of the gradient of the fused linear + logprob: the oracle's pins,
the C ABI's refusals (fake device addresses; every call returns before a HIP
call) and the binding's argument checks. No GPU needed, no kernel is launched."""
import ctypes

import numpy as np
import pytest
import torch

import datagen
import invariant_token_log_fp32_amd as rlk
from invariant_token_log_fp32_amd import VocabLayout
from oracle import linear as LIN
from oracle import linear_grad as OG

OK, NULL, ALIGN, SHAPE, GROUPS, WS = 0, -1, -2, -3, -4, -5
P = 0x10000
META = torch.device("meta")


def test_oracle_gradients_against_differences():
    """Central differences of the logprob of unrounded logits on inputs whose
    logits are exact in BF16 (so that the oracle's rounding changes nothing)."""
    hb, wb = datagen.linear_exact_inputs(5, 4, 64, 30)
    h, w = LIN.bf16_to_f64(hb), LIN.bf16_to_f64(wb)
    x = h @ w.T
    assert np.array_equal(LIN.bf16_to_f64(LIN.round_bf16(x)), x)
    t, g, tg = np.full(4, 2.0, np.float32), np.array([1.0, -0.5, 2.0, 0.0]), np.array([0, 7, 29, 3])
    gh, gw = OG.linear_logp_backward(hb, wb, 64, t, tg, g)

    def loss(h, w):
        z = h @ w.T / 2.0
        m = z.max(1, keepdims=True)
        return float((g * (z[np.arange(4), tg] - m[:, 0] - np.log(np.exp(z - m).sum(1)))).sum())

    rng = np.random.default_rng(1)
    for _ in range(5):
        dh, dw = rng.normal(0, 1, h.shape), rng.normal(0, 1, w.shape)
        e = 1e-6
        # differences of a loss of about |g| 10: rounding 1e-15 / 1e-6, curvature (e |direction|)^2
        assert abs((gh * dh).sum() - (loss(h + e * dh, w) - loss(h - e * dh, w)) / (2 * e)) < 1e-6
        assert abs((gw * dw).sum() - (loss(h, w + e * dw) - loss(h, w - e * dw)) / (2 * e)) < 1e-6
    assert not gh[3].any()


def test_oracle_leaves_rows_without_a_gradient_out():
    hb, wb = datagen.linear_exact_inputs(6, 3, 64, 20)
    hb = hb.copy()
    hb[1] = 0x7FC0
    gh, gw = OG.linear_logp_backward(hb, wb, 64, np.ones(3, np.float32), [1, 2, 3], [1.0, 0.0, 0.0])
    assert np.isfinite(gw).all() and gw.any() and not gh[1:].any()


def test_every_declared_function_is_exported():
    lib = rlk.load_library()
    names = rlk.declared_functions(rlk.TRAINING_HEADER_PATHS)
    assert {"rlk_linear_logp_backward", "rlk_linear_logp_backward_merge", "rlk_linear_logp_backward_workspace_bytes"} <= set(names)
    for n in names:
        assert hasattr(lib, n), n
        assert getattr(lib, n).argtypes is not None, n


def test_workspace_sizes():
    f = rlk.linear_logp_backward_workspace_bytes
    logits = 2 * 8192 * 152576
    assert 0 < f(8192, 4096, 152576, 151936) < logits / 2
    assert f(0, 64, 64, 64) > 0
    for n, d, vp, vr in ((-1, 64, 64, 64), ((1 << 22) + 1, 64, 64, 64), (1, 32, 64, 64), (1, 96, 64, 64), (1, 65600, 64, 64),
                         (1, 64, 100, 64), (1, 64, 64, 0), (1, 64, 64, 65), (1, 64, (1 << 22) + 64, 64)):
        assert f(n, d, vp, vr) == 0, (n, d, vp, vr)
    assert rlk.linear_logp_backward_workspace_bytes(4, 64, 64, 64, groups=3) == 0
    # no row count needs less than a smaller one
    last = 0
    for n in list(range(0, 10000, 61)) + [16384, 16385, 40000, 1 << 20, 1 << 22]:
        now = f(n, 512, 152576, 151936)
        assert now >= last, n
        last = now


def back(h=P, n=4, d=64, ldh=64, w=2 * P, ldw=64, L=None, rank=0, t=3 * P, tg=4 * P, ref=5 * P, lse=6 * P, gr=7 * P, pol=8 * P,
         state=9 * P, gp=10 * P, gh=11 * P, ldgh=64, th=0, gw=12 * P, ldgw=64, tw=0, ws=13 * P, wb=1 << 40):
    L = L if L is not None else VocabLayout(1024, 1000, 1024, 8, 1)
    return rlk.load_library().rlk_linear_logp_backward(h, n, d, ldh, w, ldw, ctypes.byref(L) if L is not False else None, rank, t, tg,
                                                       ref, lse, gr, pol, state, gp, gh, ldgh, th, gw, ldgw, tw, ws, wb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), NULL), (dict(w=None), NULL), (dict(t=None), NULL), (dict(tg=None), NULL), (dict(L=False), NULL),
    (dict(gr=None, gp=None), NULL), (dict(ref=None), NULL), (dict(lse=None), NULL), (dict(pol=None), NULL), (dict(state=None), NULL),
    (dict(gh=None, gw=None), NULL), (dict(ws=None), NULL),
    (dict(h=P + 8), ALIGN), (dict(w=P + 8), ALIGN), (dict(t=P + 2), ALIGN), (dict(tg=P + 4), ALIGN), (dict(ref=P + 2), ALIGN),
    (dict(lse=P + 1), ALIGN), (dict(gr=P + 2), ALIGN), (dict(pol=P + 2), ALIGN), (dict(state=P + 2), ALIGN), (dict(gp=P + 2), ALIGN),
    (dict(gh=P + 8), ALIGN), (dict(gw=P + 8), ALIGN), (dict(ws=P + 8), ALIGN),
    (dict(n=-1), SHAPE), (dict(n=(1 << 22) + 1), SHAPE), (dict(d=32), SHAPE), (dict(d=96), SHAPE), (dict(d=65600, ldh=65600, ldw=65600), SHAPE),
    (dict(ldh=56), SHAPE), (dict(ldh=68), SHAPE), (dict(ldh=(1 << 21) + 8), SHAPE), (dict(ldw=56), SHAPE), (dict(ldw=1 << 62), SHAPE),
    (dict(ldgh=56), SHAPE), (dict(ldgh=68), SHAPE), (dict(ldgw=0), SHAPE), (dict(ldgw=(1 << 21) + 8), SHAPE),
    (dict(th=2), SHAPE), (dict(th=-1), SHAPE), (dict(tw=3), SHAPE), (dict(rank=1), SHAPE), (dict(rank=-1), SHAPE),
    (dict(L=VocabLayout(1000, 1000, 1024, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 1025, 1024, 8, 1)), SHAPE),
    (dict(L=VocabLayout(1 << 23, 1000, 1 << 23, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 1000, 1024, 4, 1)), SHAPE),
    (dict(L=VocabLayout(1024, 1000, 1016, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 1000, 1024, 8, 3)), GROUPS), (dict(wb=1000), WS),
])
def test_backward_refuses(kw, code):
    assert back(**kw) == code


def test_no_rows_and_nothing_to_set_enqueue_nothing():
    none = dict(n=0, h=None, w=None, t=None, tg=None, ref=None, lse=None, gr=None, pol=None, state=None, gp=None)
    assert back(**none, gw=None) == OK
    assert back(**none, tw=2) == OK
    assert back(**none, gw=None, wb=0) == WS


def merge(parts=P, step=4 * 64, groups=2, n=4, d=64, out=2 * P, ld=64, kind=0):
    return rlk.load_library().rlk_linear_logp_backward_merge(parts, step, groups, n, d, out, ld, kind, None)


@pytest.mark.parametrize("kw,code", [
    (dict(parts=None), NULL), (dict(out=None), NULL), (dict(parts=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(groups=3), GROUPS),
    (dict(groups=0), GROUPS), (dict(step=255), SHAPE), (dict(step=258), SHAPE), (dict(step=1 << 62), SHAPE), (dict(n=-1), SHAPE),
    (dict(d=60), SHAPE), (dict(ld=56), SHAPE), (dict(ld=70), SHAPE), (dict(kind=2), SHAPE), (dict(n=0, parts=None, out=None, step=0), OK),
])
def test_merge_refuses(kw, code):
    assert merge(**kw) == code


def test_binding_checks_tensors():
    good = torch.empty((4, 64), dtype=torch.bfloat16, device=META)
    assert rlk._grad_out(good, (4, 64), torch.bfloat16, META, "g") is good
    for bad in (torch.empty((4, 64), dtype=torch.float16, device=META), torch.empty((4, 64), dtype=torch.bfloat16),
                torch.empty((4, 128), dtype=torch.float32, device=META)[:, ::2], torch.empty((4, 68), device=META)[:, :64],
                torch.empty((5, 64), device=META), None.__class__):
        with pytest.raises(ValueError):
            rlk._grad_out(bad, (4, 64), torch.bfloat16, META, "g")
    with pytest.raises(ValueError):
        rlk._grad_out(good, (4, 64), torch.float32, META, "g", f32_only=True)
    with pytest.raises(ValueError):  # not on a device
        rlk.linear_logp_backward(torch.zeros((4, 64), dtype=torch.bfloat16), None, 1.0, None, vocab_padded=64)
    with pytest.raises(ValueError):
        rlk.linear_logp_backward_merge(torch.zeros((2, 4, 64)))


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=META)
    with pytest.raises(ValueError, match="hidden on meta"):
        rlk.linear_logp_backward(x, x, 1.0, None, vocab_padded=64, stream=Stream())
    with pytest.raises(ValueError, match="parts on meta"):
        rlk.linear_logp_backward_merge(x, stream=Stream())
