"""The forms of the head's gradient that a trainer uses on real batches: float32 and
accumulated gradients of the projection from more than 128 rows, over launches of 8, 4, 2
and 1 shards, and ranks' parts whose shards are summed one after another, at once, and over
several launches. Tolerances as in test_gpu_linear_grad.py; where the header promises bytes,
bytes are compared."""
import numpy as np
import pytest

import invariant_token_log_fp32_amd as rlk

from gpu_util import say, to_host
from test_gpu_linear_grad import Problem, bits, close, f32, first_rows, run_all

pytestmark = pytest.mark.gpu

BUDGET = 640 << 20  # bytes that the G of several shards may take


def shards_at_once(n, vp, groups):
    """Shards of a launch: 8 / groups, halved until their G fits."""
    ldg = -(-(vp // 8) // 256) * 256
    k = 8 // groups
    while k > 1 and k * n * ldg * 2 > BUDGET:
        k //= 2
    return k


def cost(n, d, shards):
    """Cost of grad_hidden's tiles (rounds over 256 compute units) as the kernel takes them."""
    def tiles(bm, bn):
        return -(-n // bm) * -(-d // bn) * shards

    def rounds(t):
        return -(-t // 256)

    large = tiles(256, 256)
    best = rounds(large) * 100
    for bm, bn, each, parts in ((128, 256, 70, 2), (128, 128, 44, 4), (64, 128, 30, 8)):
        best = min(best, rounds(tiles(bm, bn)) * each)
        if large >= 256:
            best = min(best, large // 256 * 100 + rounds(large % 256 * parts) * each)
    return best


def in_turn(n, d, shards):
    return cost(n, d, 1) * shards <= cost(n, d, shards)


@pytest.mark.parametrize("n,d,vr,vp", [(129, 320, 2500, 2560), (257, 256, 1111, 1152), (300, 1088, 700, 1024), (640, 192, 900, 960)])
@pytest.mark.parametrize("terms", ["ref", "both"])
def test_accumulated_and_float32_against_the_oracle(n, d, vr, vp, terms):
    import torch
    say(f"case: {n} x {d} x {vr}, {terms}")
    p = Problem(n + d, n, d, vr, vp, temps=(0.7, 1.0, 0.0, 1.3), top_p=1.0 if terms == "ref" else 0.9)
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want(terms)
    hidden, plain = torch.empty((n, d), device="cuda:0"), torch.empty((vr, d), device="cuda:0")
    gh, gw = run_all(p, terms, grad_hidden=hidden, grad_weight=plain)
    close(gh, want_h, mag_h, extra_h, vr, False, "grad_hidden")
    close(gw, want_w, mag_w, extra_w, n, False, "grad_weight")
    before = torch.randn((vr, d), device="cuda:0")
    wide = torch.full((vr + 1, d + 24), 7.0, device="cuda:0")
    wide[:vr, :d] = before
    run_all(p, terms, grad_weight=wide[:vr, :d], accumulate=True)
    assert torch.equal(wide[:vr, :d], before + plain)  # one float32 addition
    assert bool((wide[vr:] == 7.0).all()) and bool((wide[:, d:] == 7.0).all()), "written outside the gradient"
    short = run_all(p, terms)
    assert np.array_equal(bits(short[0]), bits(gh.to(torch.bfloat16))) and np.array_equal(bits(short[1]), bits(plain.to(torch.bfloat16)))


def test_accumulated_over_several_launches():
    """Two micro-batches into one gradient, at 8, 4, 2 and 1 shards a launch."""
    import torch
    say("case: up to 9000 rows of a 151936 x 64 head")
    p = Problem(22, 9000, 64, 151936, 152576)
    seen = set()
    for n in (500, 2600, 5000, 9000):
        say(f"  {n} rows")
        seen.add(shards_at_once(n, p.vp, 1))
        a, kw = first_rows(p, n, n)
        plain = rlk.linear_logp_backward(*a, **kw, grad_weight=torch.empty((p.vr, p.d), device="cuda:0"))[1]
        assert np.array_equal(bits(rlk.linear_logp_backward(*a, **kw)[1]), bits(plain.to(torch.bfloat16)))
        total = torch.randn((p.vr, p.d), device="cuda:0")
        want = (total + plain) + plain
        for _ in range(2):
            got = rlk.linear_logp_backward(*a, **kw, grad_weight=total, accumulate=True)[1]
        assert got is total and torch.equal(total, want)
    assert seen == {8, 4, 2, 1}


def ranks(p, a, kw, groups, whole):
    """Every rank's part and their merge against the whole's bytes."""
    import torch
    gh, gw, gh32 = whole
    cols = p.vp // groups
    parts = torch.full((groups, a[0].shape[0], p.d), 7.0, device="cuda:0")
    for rank in range(groups):
        lo, hi = min(p.vr, rank * cols), min(p.vr, (rank + 1) * cols)
        _, wg = rlk.linear_logp_backward(a[0], p.w[lo:hi], *a[2:], **kw, vocab_real=p.vr, rank=rank, groups=groups,
                                         grad_hidden=parts[rank])
        assert np.array_equal(bits(wg), bits(gw)[lo:hi]), f"grad_weight of rank {rank} of {groups}"
    assert np.array_equal(bits(rlk.linear_logp_backward_merge(parts)), bits(gh)), f"grad_hidden at {groups} ranks"
    merged = rlk.linear_logp_backward_merge(parts, out=torch.empty_like(gh32))
    assert np.array_equal(bits(merged), bits(gh32)), f"float32 grad_hidden at {groups} ranks"


def whole_of(a, kw):
    import torch
    gh, gw = rlk.linear_logp_backward(*a, **kw)
    gh32, _ = rlk.linear_logp_backward(*a, **kw, weight_grad=False, grad_hidden=torch.empty(gh.shape, device="cuda:0"))
    assert np.array_equal(bits(gh), bits(gh32.to(torch.bfloat16)))
    return gh, gw, gh32


def test_ranks_that_sum_their_shards_one_after_another():
    """All rows live; a part of them, few enough for one round of tiles a shard; so few that
    the device sums at once where the host has planned for sums in turn."""
    import torch
    n, d, vr, vp = 8192, 4032, 1000, 1024
    say(f"case: {n} x {d} x {vr}")
    p = Problem(31, n, d, vr, vp)
    a, kw = p.args()
    every = None
    for live, turn in ((8192, True), (4000, True), (2000, False)):
        say(f"  {live} rows with a gradient")
        for k in (8, 4, 2):
            assert shards_at_once(n, vp, 8 // k) == k and in_turn(n, d, k) and in_turn(live, d, k) == turn
        keep = np.zeros(n, bool)
        keep[np.random.default_rng(live).permutation(n)[:live]] = True
        kw["grad_ref"] = f32(np.where(keep, p.g_ref, 0))
        whole = whole_of(a, kw)
        if every is None:
            every = whole
        assert np.array_equal(bits(whole[0])[keep], bits(every[0])[keep]) and not bits(whole[0])[~keep].any()
        for groups in (2, 4, 8):
            ranks(p, a, kw, groups, whole)


@pytest.mark.parametrize("n,at_once", [(2600, {1: 4, 2: 4, 4: 2, 8: 1}), (5000, {1: 2, 2: 2, 4: 2, 8: 1}), (9000, {1: 1, 2: 1, 4: 1, 8: 1})])
def test_ranks_over_several_launches(n, at_once):
    say(f"case: {n} rows of a 151936 x 64 head")
    p = Problem(25, n, 64, 151936, 152576)
    assert {g: shards_at_once(n, p.vp, g) for g in (1, 2, 4, 8)} == at_once
    a, kw = p.args()
    whole = whole_of(a, kw)
    for groups in (2, 4, 8):
        ranks(p, a, kw, groups, whole)
