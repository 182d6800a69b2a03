"""The training head's operators as a trainer runs them: norm, fused linear +
logprob, its gradient, the norm's backward, the gradient norm. Every stage is held
to its oracle on what the stage before it left on the device."""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import l2norm as OL
from oracle import layer_norm as LN
from oracle import linear as LIN
from oracle import linear_grad as OG

from gpu_util import TOL, assert_close, say, to_host

pytestmark = pytest.mark.gpu


def host_bits(t):
    import torch
    return to_host(t.contiguous().view(torch.int16)).view(np.uint16)


@pytest.mark.parametrize("rms", [True, False])
def test_a_training_step_of_the_head(rms):
    import torch
    say(f"case: the head's forward and backward, rms {rms}")
    rng = np.random.default_rng(11)
    n, d, vr, vp = 200, 320, 1500, 1536
    stream32 = torch.from_numpy(rng.normal(0.1, 3, (n, d)).astype(np.float32)).to("cuda:0")
    gain = torch.from_numpy(rng.normal(1, 0.1, d).astype(np.float32)).to("cuda:0")
    wb = datagen.f32_to_bf16_bits(rng.normal(0, 2 / np.sqrt(d), (vr, d)).astype(np.float32))
    head = torch.from_numpy(wb.view(np.int16)).to("cuda:0").view(torch.bfloat16)
    target = torch.from_numpy(rng.integers(0, vr, n)).to("cuda:0")
    t = torch.full((n,), 0.9, device="cuda:0")
    advantage = rng.normal(0, 1, n).astype(np.float32)
    advantage[rng.random(n) < 0.3] = 0  # prompt tokens
    up = torch.from_numpy(advantage).to("cuda:0")

    hidden, mean, rstd = rlk.layer_norm(stream32, gain, rms=rms, return_stats=True)
    logp, lse = rlk.linear_logp(hidden, head, t, target, vocab_padded=vp, return_lse=True)
    gh, gw = rlk.linear_logp_backward(hidden, head, t, target, vocab_padded=vp, ref_logp=logp, lse=lse, grad_ref=up,
                                      grad_weight=torch.empty((vr, d), device="cuda:0"))
    dx, dgain, _ = rlk.layer_norm_backward(gh, stream32, gain, mean, rstd, rms=rms)
    sumsq, norm = rlk.l2norm([gw, dgain])

    hb = host_bits(hidden)
    temps = np.full(n, 0.9, np.float32)
    want_logp, _ = LIN.linear_logp(hb, wb, vp, temps, to_host(target))
    # the oracle rounds logits from float64 sums: where a float32 sum falls on the other
    # side of the middle the logprob moves by up to half a BF16 step of a logit below 16
    off = np.abs(to_host(logp) - want_logp)
    assert (off <= 2.0 ** -4 / 0.9 + TOL).all() and np.median(off) <= TOL
    logits = host_bits(rlk.linear(hidden, head, vocab_padded=vp))
    G = OG.logit_grad(logits, vr, temps, to_host(target), advantage)
    want_h, want_w, _, _ = OG.products(G, hb, wb)
    for got, want, what, most in ((gh, want_h, "grad_hidden", 4e-3), (gw, want_w, "grad_weight", 3e-3)):
        # half a BF16 step of G (2^-8 at most, 2^-9.8 as a root mean square) and of the output
        rel = np.linalg.norm(to_host(got.double()) - want) / np.linalg.norm(want)
        say(f"  {what}: relative error {rel:.2e}")
        assert rel <= most, what
    x = to_host(stream32).astype(np.float64)
    ghv = LIN.bf16_to_f64(host_bits(gh))
    want_dx, want_dgain, _ = LN.backward(ghv, x, to_host(gain), to_host(mean) if not rms else np.zeros(n), to_host(rstd), rms)
    assert np.linalg.norm(to_host(dx) - want_dx) <= 1e-6 * np.linalg.norm(want_dx)
    assert np.linalg.norm(to_host(dgain) - want_dgain) <= 1e-6 * np.linalg.norm(want_dgain)
    assert not to_host(dx)[advantage == 0].any()
    want_sumsq, want_norm = OL.norm([to_host(gw).ravel(), to_host(dgain)])
    assert float(sumsq.item()) == want_sumsq and float(norm.item()) == want_norm


def test_the_step_in_one_graph():
    """Captured once and replayed on other hidden states, against eager calls."""
    import torch
    say("case: the step as a graph")
    rng = np.random.default_rng(12)
    n, d, vr, vp = 130, 256, 900, 960
    dev = "cuda:0"
    x = torch.from_numpy(rng.normal(0, 1, (n, d)).astype(np.float32)).to(dev)
    gain = torch.ones(d, device=dev)
    head = torch.from_numpy(rng.normal(0, 0.1, (vr, d)).astype(np.float32)).to(dev).to(torch.bfloat16)
    target = torch.from_numpy(rng.integers(0, vr, n)).to(dev)
    t, up = torch.ones(n, device=dev), torch.from_numpy(rng.normal(0, 1, n).astype(np.float32)).to(dev)
    bf, f32 = torch.bfloat16, torch.float32
    o = dict(h=torch.empty((n, d), dtype=bf, device=dev), mean=torch.empty(n, device=dev), rstd=torch.empty(n, device=dev),
             lp=torch.empty(n, device=dev), lse=torch.empty(n, device=dev), gh=torch.empty((n, d), dtype=bf, device=dev),
             gw=torch.empty((vr, d), dtype=bf, device=dev), dx=torch.empty((n, d), device=dev), dg=torch.empty(d, device=dev))
    ws = [torch.empty(k, dtype=torch.uint8, device=dev) for k in
          (rlk.linear_logp_workspace_bytes(n, vp, vr), rlk.linear_logp_backward_workspace_bytes(n, d, vp, vr),
           rlk.layer_norm_backward_workspace_bytes(n, d))]

    def step(o):
        rlk.layer_norm(x, gain, return_stats=True, out=o["h"], mean_out=o["mean"], rstd_out=o["rstd"])
        rlk.linear_logp(o["h"], head, t, target, vocab_padded=vp, out=o["lp"], lse_out=o["lse"], workspace=ws[0])
        rlk.linear_logp_backward(o["h"], head, t, target, vocab_padded=vp, ref_logp=o["lp"], lse=o["lse"], grad_ref=up, grad_hidden=o["gh"],
                                 grad_weight=o["gw"], workspace=ws[1])
        rlk.layer_norm_backward(o["gh"], x, gain, o["mean"], o["rstd"], grad_x=o["dx"], grad_weight=o["dg"], workspace=ws[2])

    step(o)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(o)
    for k in range(3):
        x.copy_(torch.from_numpy(rng.normal(0, 1 + k, (n, d)).astype(np.float32)))
        want = {key: torch.empty_like(v) for key, v in o.items()}
        step(want)
        torch.cuda.synchronize()
        for v in o.values():
            v.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        for key in o:
            assert torch.equal(o[key], want[key]), (k, key)
