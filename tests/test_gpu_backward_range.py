"""rlk_logp_backward on rows that have a policy term and no reference term, at logits
beyond the range of float32 exponentials (x / T above 88): the absent term adds nothing,
whatever the size of the logits and whatever stands in its statistics.

Tolerances as in test_gpu_backward.py.
"""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import logp as O

from gpu_util import say, to_host, upload, upload_logits
from test_gpu_backward import bits_to_f64, compare_row, grad_tolerance

pytestmark = pytest.mark.gpu

N, VP, VR = 12, 1024, 1000


def rows(seed, top):
    """(logit bits [N, VP], temperatures, targets): the largest scaled logit of each row is about `top`."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2.0, (N, VP)).astype(np.float32)
    temps = rng.choice(np.asarray([0.1, 0.7, 1.0], np.float32), N)
    x += (top * temps - x.max(1))[:, None].astype(np.float32)  # a common offset: the distributions stay wide
    bits = datagen.f32_to_bf16_bits(x)
    bits[:, VR:] = 0xFF80  # -inf
    order = np.argsort(-bits_to_f64(bits)[:, :VR], axis=1, kind="stable")
    targets = order[np.arange(N), np.where(np.arange(N) % 4 == 3, VR - 1, np.arange(N) % 4)]  # every fourth outside its support
    return bits, temps, targets.astype(np.int64)


@pytest.mark.parametrize("top", [60.0, 130.0, 900.0])
@pytest.mark.parametrize("form", ["absent", "zero", "zero, statistics unset"])
def test_the_policy_term_alone(top, form):
    import torch
    say(f"case: scaled logits up to {top}, reference term {form}")
    bits, temps, targets = rows(int(top), top)
    lg, t, tg = upload_logits(bits), upload(temps, torch.float32), upload(targets, torch.int64)
    pol, ref, lse, state = rlk.logp_nucleus(lg, t, 0.9, -1, tg, vocab_real=VR, return_state=True)
    g_pol = np.linspace(-2, 2, N).astype(np.float32)
    kw = dict(policy_logp=pol, support_state=state, grad_policy=upload(g_pol, torch.float32))
    if form != "absent":
        kw.update(ref_logp=ref, lse=torch.full_like(lse, float("nan")) if "unset" in form else lse, grad_ref=torch.zeros_like(lse))
    got = to_host(rlk.logp_backward(lg, t, tg, vocab_real=VR, **kw).view(torch.int16)).view(np.uint16)
    lse_s, thr, status = (to_host(a) for a in rlk.support_state_fields(state))
    assert set(status.tolist()) == {0, 1}, "both kinds of target are reached"
    pol_h = to_host(pol)
    for i in range(N):
        T, target = float(temps[i]), int(targets[i])
        pol_o, ref_o, info = O.nucleus_row(bits[i], VR, T, 0.9, -1, target, want_mask=True)
        if info.ambiguous:  # the support may differ by one boundary class
            continue
        _, lse_o = O.ref_logp_row(bits[i], VR, T, target)
        want = O.grad_row(bits[i], VP, VR, T, target, 0.0, float(g_pol[i]), 0.9, -1)
        assert np.isfinite(want).all()
        g_p = float(g_pol[i]) if status[i] == 1 else 0.0
        tol = grad_tolerance(bits[i], VP, VR, T, target, 0.0, g_p, lse_o, lse_o, ref_o, ref_o, pol_o, float(pol_h[i]),
                             info.lse_support, float(lse_s[i]), info.support_mask, want, bits_to_f64(got[i]))
        compare_row(got[i], want, tol, f"row {i}")
        if g_p == 0.0:
            assert (bits_to_f64(got[i]) == 0).all(), f"row {i}: a target outside the support has no gradient"


@pytest.mark.parametrize("targets", ["any", "the likeliest"])
def test_the_gradient_of_kept_logits_and_of_the_fused_linear_agree_there(targets):
    """An identity times 4 as hidden states: grad_weight holds 4 G^T. Of these logits a
    support holds a few columns: any target lies outside it, the likeliest inside."""
    import torch
    n, d, vr, vp = 64, 64, 500, 512
    say(f"case: {n} rows of {vr} logits up to some hundreds, policy term alone, targets: {targets}")
    rng = np.random.default_rng(3)
    w = torch.from_numpy((30 + rng.normal(0, 2, (vr, d))).astype(np.float32)).to("cuda:0").to(torch.bfloat16)
    h = torch.eye(n, d, dtype=torch.bfloat16, device="cuda:0") * 4
    t = upload(rng.choice(np.asarray([0.3, 1.0], np.float32), n), torch.float32)
    tg = upload(rng.integers(0, vr, n), torch.int64)
    logits = rlk.linear(h, w, vocab_padded=vp)
    if targets == "the likeliest":
        tg = logits[:, :vr].float().argmax(1)
    pol, _, _, state = rlk.logp_nucleus(logits, t, 0.95, -1, tg, vocab_real=vr, return_state=True)
    assert bool((state[:, 2] == (targets == "the likeliest")).all())
    assert float(logits[:, :vr].float().abs().max()) > 130
    kw = dict(policy_logp=pol, support_state=state, grad_policy=upload(rng.normal(0, 1, n), torch.float32))
    G = rlk.logp_backward(logits, t, tg, vocab_real=vr, **kw)
    _, gw = rlk.linear_logp_backward(h, w, t, tg, vocab_padded=vp, hidden_grad=False, **kw)
    assert bool(G.isfinite().all())
    if targets == "any":
        assert not G.any()
    assert bool((gw == (G[:, :vr].float() * 4).to(torch.bfloat16).T).all())
