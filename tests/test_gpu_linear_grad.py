"""GPU parity of the gradient of the fused linear + logprob against the float64
oracle (oracle/linear_grad.py), and the properties that its header states.

Tolerances. G, the gradient of a BF16 logit, is rounded to BF16 (2^-8 of its
value) from a float32 value whose exponent argument x c - lse log2 e is off by at
most 2^-22 of |x| / T + |lse| (two roundings each) and whose lse is off by 2e-5:
with |x| / T and |lse| below 64, less than 6e-5; together `G_REL`. A sum over n
products is off by at most G_REL of the sum of the magnitudes, and 2^-23 of it
for each matrix instruction or addition (a whole unit: the order inside an
instruction is not specified); a BF16 output adds 2^-8 of the value.
The target's G is -g expm1(ref) / T with the forward's float32 logprob, off by at
most 2e-5: d/dref of it is -g exp(ref) / T, at most g / T in magnitude, so it is
off by up to 2e-5 |g| / T however small it is itself (rows whose target holds
nearly all of the mass). That adds 2e-5 |g| / T of the target's row of the
projection, and of the row's hidden states in the target's row of grad_weight.
The logits themselves are the bits that rlk_linear writes, so the oracle takes
those and no rounding of a logit can fall differently.
"""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import linear as LIN
from oracle import linear_grad as OG

from gpu_util import say, to_host

pytestmark = pytest.mark.gpu

G_REL = 2.0 ** -8 + 6e-5


def upload(bits, pad=0, fill=0x7FC0):
    import torch
    n, d = bits.shape
    buf = np.full((n, d + pad), fill, dtype=np.uint16)
    buf[:, :d] = bits
    return torch.from_numpy(buf.view(np.int16)).to("cuda:0").view(torch.bfloat16)[:, :d]


def f32(v):
    import torch
    return torch.as_tensor(np.ascontiguousarray(v), dtype=torch.float32, device="cuda:0")


class Problem:
    """Inputs on the device and what the forward calls leave of them."""

    def __init__(self, seed, n, d, vr, vp, *, temps=(0.7, 1.0, 1.3), top_p=1.0, hpad=0, wpad=0, lean=2.0):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.d, self.vr, self.vp, self.top_p = n, d, vr, vp, top_p
        w = rng.normal(0, 2.5 / np.sqrt(d), (vr, d))
        self.target = rng.integers(0, vr, n)
        h = rng.normal(0, 1, (n, d)) + lean * rng.random((n, 1)) * w[self.target]
        self.hb = datagen.f32_to_bf16_bits(h.astype(np.float32))
        self.wb = datagen.f32_to_bf16_bits(w.astype(np.float32))
        self.h, self.w = upload(self.hb, hpad), upload(self.wb, wpad)
        self.temps = rng.choice(np.asarray(temps, np.float32), n)
        self.t = f32(self.temps)
        self.tg = torch.from_numpy(self.target).to("cuda:0")
        self.g_ref = rng.normal(0, 1, n).astype(np.float32)
        self.g_pol = rng.normal(0, 1, n).astype(np.float32)
        self.forward()

    def forward(self):
        self.logits = rlk.linear(self.h, self.w, vocab_padded=self.vp)
        self.pol, self.ref, self.lse, self.state = rlk.logp_nucleus(self.logits, self.t, self.top_p, -1, self.tg,
                                                                    vocab_real=self.vr, return_state=True)

    def args(self, terms="ref", rows=slice(None)):
        host = rows if isinstance(rows, slice) else rows.cpu().numpy()
        kw = dict(vocab_padded=self.vp)
        if terms != "policy":
            kw.update(ref_logp=self.ref[rows].contiguous(), lse=self.lse[rows].contiguous(), grad_ref=f32(self.g_ref[host]))
        if terms != "ref":
            kw.update(policy_logp=self.pol[rows].contiguous(), support_state=self.state[rows].contiguous(),
                      grad_policy=f32(self.g_pol[host]))
        return (self.h[rows], self.w, self.t[rows].contiguous(), self.tg[rows].contiguous()), kw

    def want(self, terms="ref"):
        bits = to_host(self.logits.view(__import__("torch").int16)).view(np.uint16)
        G = OG.logit_grad(bits, self.vr, self.temps, self.target, None if terms == "policy" else self.g_ref,
                          None if terms == "ref" else self.g_pol, self.top_p)
        want_h, want_w, mag_h, mag_w = OG.products(G, self.hb, self.wb)
        w, h = np.abs(LIN.bf16_to_f64(self.wb)), np.abs(LIN.bf16_to_f64(self.hb))
        up = (np.abs(self.g_ref) * (terms != "policy") + np.abs(self.g_pol) * (terms != "ref")).astype(np.float64)
        live = (up != 0) & (self.temps > 0)  # a support of the target alone has G = 0 here, and 2e-5 |g| / T at most there
        at_target = np.where(live, 2e-5 * up / np.where(self.temps > 0, self.temps, 1.0), 0.0)
        extra_h = at_target[:, None] * w[self.target]
        extra_w = np.zeros_like(mag_w)
        np.add.at(extra_w, self.target[live], (at_target[:, None] * h)[live])
        return want_h, want_w, mag_h, mag_w, extra_h, extra_w


def close(got, want, mag, extra, n_terms, bf16, what):
    got = to_host(got.double())
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    off = np.abs(got - want)
    tol = mag * (G_REL + (n_terms / 16 + 16) * 2.0 ** -23) + extra + (2.0 ** -8 * np.abs(want) if bf16 else 0.0) + 1e-30
    bad = ~(off <= tol) & ~np.isnan(want)
    assert not bad.any(), f"{what}: off by {off[bad].max():.3e} at {np.argwhere(bad)[:4].tolist()}, {bad.sum()} of {bad.size}"
    norm = np.linalg.norm(np.nan_to_num(want))
    if norm and not np.isnan(want).any():
        rel = np.linalg.norm(off) / norm
        say(f"  {what}: relative error {rel:.2e}")


SIZES = [(1, 64, 300, 320), (2, 128, 1000, 1024), (5, 192, 64, 64), (37, 320, 2500, 2560), (257, 256, 1111, 1152),
         (300, 1088, 700, 1024), (64, 64, 4096, 4096), (130, 576, 5000, 8192), (513, 128, 2049, 2112),
         (64, 832, 3000, 3136), (65, 64, 1000, 1024), (128, 320, 2111, 2176), (129, 128, 600, 640), (640, 192, 900, 960),
         (1025, 64, 500, 512)]


@pytest.mark.parametrize("n,d,vr,vp", SIZES)
@pytest.mark.parametrize("terms", ["ref", "both"])
def test_matches_the_oracle(n, d, vr, vp, terms):
    say(f"case: {n} x {d} x {vr} of {vp}, {terms}")
    p = Problem(n + d, n, d, vr, vp, temps=(0.7, 1.0, 0.0, 1.3), top_p=1.0 if terms == "ref" else 0.9)
    a, kw = p.args(terms)
    gh, gw = rlk.linear_logp_backward(*a, **kw)
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want(terms)
    close(gh, want_h, mag_h, extra_h, vr, True, "grad_hidden")
    close(gw, want_w, mag_w, extra_w, n, True, "grad_weight")


@pytest.mark.parametrize("n", [1, 64, 128, 200, 256, 513])
@pytest.mark.parametrize("vr,vp", [(201, 256), (2049, 2112), (1, 64)])
def test_the_last_column_of_an_odd_vocabulary(n, vr, vp):
    """Every row's target is the last column, whose place in its shard is odd: the
    largest part of G lies in half a word at the end of each row."""
    import torch
    say(f"case: {n} rows, last column of {vr}")
    p = Problem(n, n, 128, vr, vp, temps=(1.0,), lean=0.0)
    p.target[:] = vr - 1
    p.tg = torch.from_numpy(p.target).to("cuda:0")
    p.forward()
    gh, gw = run_all(p)
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want()
    close(gh, want_h, mag_h, extra_h, vr, True, "grad_hidden")
    close(gw, want_w, mag_w, extra_w, n, True, "grad_weight")


def run_all(p, terms="ref", **more):
    a, kw = p.args(terms)
    kw.update(more)
    return rlk.linear_logp_backward(*a, **kw)


def bits(t):
    import torch
    return to_host(t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("top_p", [0.5, 0.95])
def test_the_policy_term_alone_and_what_it_does_not_read(top_p):
    say(f"case: policy term alone, top-p {top_p}")
    p = Problem(5, 41, 256, 900, 1024, top_p=top_p, lean=1.0)
    a, kw = p.args("policy")
    gh, gw = rlk.linear_logp_backward(*a, **kw)
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want("policy")
    close(gh, want_h, mag_h, extra_h, p.vr, True, "grad_hidden")
    close(gw, want_w, mag_w, extra_w, p.n, True, "grad_weight")
    assert (to_host(p.state)[:, 2] == 0).any(), "no target outside its support: the case is not reached"


def test_large_logits_without_a_reference_term():
    """|x| / T beyond the range of float32 exponentials: the absent term must not turn 0 x inf into NaN."""
    say("case: logits of some hundreds")
    p = Problem(6, 9, 128, 500, 512, temps=(0.1,), top_p=0.9, lean=0.0)
    p.h.mul_(4)
    p.hb = to_host(p.h.view(__import__("torch").int16)).view(np.uint16)
    p.forward()
    assert float(p.logits[:, :p.vr].float().abs().max()) / 0.1 > 130
    gh, gw = run_all(p, "policy")
    assert bool(gh.isfinite().all()) and bool(gw.isfinite().all())


@pytest.mark.parametrize("hidden_type", ["bfloat16", "float32"])
@pytest.mark.parametrize("weight_type", ["bfloat16", "float32", "add"])
def test_types_strides_and_what_lies_around(hidden_type, weight_type):
    import torch
    say(f"case: grad_hidden {hidden_type}, grad_weight {weight_type}, wider rows")
    p = Problem(7, 70, 320, 1500, 1536, hpad=8, wpad=24)
    dev = p.h.device
    gh = torch.full((p.n + 1, p.d + 16), 7.0, dtype=getattr(torch, hidden_type), device=dev)
    wt = torch.float32 if weight_type == "add" else getattr(torch, weight_type)
    gw = torch.full((p.vr + 1, p.d + 8), 7.0, dtype=wt, device=dev)
    before = torch.randn((p.vr, p.d), device=dev)
    if weight_type == "add":
        gw[:p.vr, :p.d] = before
    a, kw = p.args()
    out = rlk.linear_logp_backward(*a, **kw, grad_hidden=gh[:p.n, :p.d], grad_weight=gw[:p.vr, :p.d], accumulate=weight_type == "add")
    assert out[0].data_ptr() == gh.data_ptr() and out[1].data_ptr() == gw.data_ptr()
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want()
    if weight_type == "add":
        want_w = want_w + to_host(before.double())
        extra_w = extra_w + 2.0 ** -24 * np.abs(want_w)  # one float32 addition
    close(gh[:p.n, :p.d], want_h, mag_h, extra_h, p.vr, hidden_type == "bfloat16", "grad_hidden")
    close(gw[:p.vr, :p.d], want_w, mag_w, extra_w, p.n, weight_type == "bfloat16", "grad_weight")
    for t, r in ((gh, p.n), (gw, p.vr)):
        assert bool((t[r:] == 7.0).all()) and bool((t[:, p.d:] == 7.0).all()), "written outside the gradient"


def test_one_output_alone_is_the_same():
    say("case: one output alone")
    p = Problem(8, 77, 192, 777, 1024)
    gh, gw = run_all(p)
    h1, none = run_all(p, weight_grad=False)
    assert none is None and np.array_equal(bits(h1), bits(gh))
    none, w1 = run_all(p, hidden_grad=False)
    assert none is None and np.array_equal(bits(w1), bits(gw))


def test_rows_without_a_gradient_are_left_out():
    """Their hidden states, temperatures, targets and statistics are NaN or out of
    range; the bytes of all else are those of the call without them."""
    import torch
    say("case: masked rows that hold NaN")
    p = Problem(9, 300, 256, 1200, 1216, top_p=0.9)
    keep = np.random.default_rng(1).random(p.n) < 0.4
    idx = np.flatnonzero(keep)
    at = torch.from_numpy(idx).to("cuda:0")
    a, kw = p.args("both", rows=at)
    gh0, gw0 = rlk.linear_logp_backward(*a, **kw)
    off = torch.from_numpy(~keep).to("cuda:0")
    p.g_ref[~keep] = 0
    p.g_pol[~keep] = 0
    p.h[off] = float("nan")
    p.t[off] = float("nan")
    p.tg[off] = -5
    for v in (p.ref, p.lse, p.pol):
        v[off] = float("nan")
    p.state[off] = -2
    gh, gw = run_all(p, "both")
    assert np.array_equal(bits(gh)[idx], bits(gh0)) and np.array_equal(bits(gw), bits(gw0))
    assert (bits(gh)[~keep] == 0).all()


def test_no_row_has_a_gradient():
    import torch
    say("case: no gradient at all")
    p = Problem(10, 65, 128, 600, 640)
    p.g_ref[:] = 0
    gw = torch.full((p.vr, p.d), 3.0, device="cuda:0")
    gh, _ = run_all(p, grad_weight=gw, accumulate=True)
    assert not gh.any() and bool((gw == 3.0).all())
    gh, gw = run_all(p)
    assert not gh.any() and not gw.any()
    p.t.zero_()  # greedy rows: the logprob is piecewise constant
    p.g_ref[:] = 1
    gh, gw = run_all(p)
    assert not gh.any() and not gw.any()


def test_no_rows():
    import torch
    say("case: no rows")
    p = Problem(11, 4, 128, 600, 640)
    a, kw = p.args(rows=slice(0, 0))
    gw = torch.full((p.vr, p.d), 3.0, device="cuda:0")
    gh, _ = rlk.linear_logp_backward(*a, **kw, grad_weight=gw, accumulate=True)
    assert tuple(gh.shape) == (0, p.d) and bool((gw == 3.0).all())
    gh, gw2 = rlk.linear_logp_backward(*a, **kw, grad_weight=gw)
    assert bool((gw == 0).all())


@pytest.mark.parametrize("what", ["temperature", "target", "reference"])
def test_an_invalid_row_is_nan_and_so_is_the_projections_gradient(what):
    say(f"case: invalid {what}")
    p = Problem(12, 40, 128, 500, 512)
    {"temperature": p.t, "target": p.tg, "reference": p.ref}[what][17] = {"temperature": -1.0, "target": 500, "reference": float("nan")}[what]
    gh, gw = run_all(p)
    nan = to_host(gh.isnan())
    assert nan[17].all() and not np.delete(nan, 17, 0).any()
    assert bool(gw.isnan().all())


@pytest.mark.parametrize("n,vr,vp", [(300, 2000, 2048), (5, 152, 1024)])
def test_bytes_do_not_depend_on_the_batch(n, vr, vp):
    import torch
    say(f"case: batches of {n}")
    p = Problem(13, n, 256, vr, vp, top_p=0.9)
    gh, _ = run_all(p, "both")
    order = torch.from_numpy(np.random.default_rng(3).permutation(n)).to("cuda:0")
    for rows in (order, torch.arange(1, device="cuda:0"), torch.arange(n // 2, n // 2 + 2, device="cuda:0")):
        a, kw = p.args("both", rows=rows)
        pick = rows.cpu().numpy()
        got, _ = rlk.linear_logp_backward(*a, **kw)
        assert np.array_equal(bits(got), bits(gh)[pick])


def first_rows(p, k, n):
    """Arguments of a call with p's first n rows, of which the first k have a gradient."""
    import torch
    a, kw = p.args(rows=torch.arange(n, device="cuda:0"))
    up = kw["grad_ref"].clone()
    up[k:] = 0.0
    return a, dict(kw, grad_ref=up)


# Heads and row counts whose products take tiles of every size (64 and 128 x 128, 128 and
# 256 x 256) and whole rounds of the largest with the rest cut into each smaller one, sum
# grad_hidden's shards all at once and one after another, and have odd ends of rows,
# columns and K in each.
@pytest.mark.parametrize("d,vr,vp,rows", [(1024, 20000, 20032, (3, 100, 201, 300, 520, 1101)),
                                          (1088, 13999, 14336, (129, 190, 700)), (2048, 19999, 20032, (130, 385, 641)),
                                          (4096, 1000, 1024, (2, 300, 4096)), (1088, 20000, 20032, (200, 801, 1601)),
                                          (1088, 13999, 14336, (128, 1101, 1401)), (2048, 20000, 20032, (150, 1101, 1401))])
def test_bytes_do_not_depend_on_the_tiles(d, vr, vp, rows):
    n = max(rows)
    say(f"case: rows {rows} of a {vr} x {d} head")
    p = Problem(21, n, d, vr, vp)
    a, kw = first_rows(p, n, n)
    whole, _ = rlk.linear_logp_backward(*a, **kw)
    whole = bits(whole)
    for k in rows:
        say(f"  {k} rows")
        a, kw = first_rows(p, k, k)
        gh, gw = rlk.linear_logp_backward(*a, **kw)
        assert np.array_equal(bits(gh), whole[:k])
        if k < n:
            a, kw = first_rows(p, k, n)
            mh, mw = rlk.linear_logp_backward(*a, **kw)
            assert np.array_equal(bits(mh)[:k], whole[:k]) and not bits(mh)[k:].any()
            assert np.array_equal(bits(mw), bits(gw))


def test_a_long_head_against_the_oracle():
    say("case: 201 rows of a 20000 x 1024 head")
    p = Problem(21, 201, 1024, 20000, 20032)
    gh, gw = run_all(p)
    want_h, want_w, mag_h, mag_w, extra_h, extra_w = p.want()
    close(gh, want_h, mag_h, extra_h, 20000, True, "grad_hidden")
    close(gw, want_w, mag_w, extra_w, 201, True, "grad_weight")


def test_bytes_do_not_depend_on_how_many_shards_a_launch_takes():
    """8, 4, 2 and 1 shards of logits in the workspace at a time."""
    say("case: 9000 rows of a 151936 x 64 head")
    p = Problem(22, 9000, 64, 151936, 152576)
    a, kw = first_rows(p, 9000, 9000)
    whole = bits(rlk.linear_logp_backward(*a, **kw)[0])
    a, kw = first_rows(p, 500, 500)
    gh, gw = rlk.linear_logp_backward(*a, **kw)
    assert np.array_equal(bits(gh), whole[:500])
    for n in (2600, 5000, 9000):
        say(f"  {n} rows")
        a, kw = first_rows(p, 500, n)
        mh, mw = rlk.linear_logp_backward(*a, **kw)
        assert np.array_equal(bits(mh)[:500], whole[:500]) and not bits(mh)[500:].any()
        assert np.array_equal(bits(mw), bits(gw))


@pytest.mark.parametrize("n", [2150, 4250, 8400, 9000])
def test_the_same_bytes_every_time(n):
    """A narrow head, whose loads come from the caches: they are soon there, also where a
    wave of the workgroup is late (its code is read for the first time)."""
    say(f"case: {n} rows of a 151936 x 64 head, again and again")
    p = Problem(24, n, 64, 151936, 152576)
    a, kw = first_rows(p, n, n)
    gh, gw = rlk.linear_logp_backward(*a, **kw)
    for _ in range(10):
        mh, mw = rlk.linear_logp_backward(*a, **kw)
        assert np.array_equal(bits(mh), bits(gh)) and np.array_equal(bits(mw), bits(gw))
    a, kw = first_rows(p, 64, 64)
    assert np.array_equal(bits(rlk.linear_logp_backward(*a, **kw)[0]), bits(gh)[:64])


def test_strides_whose_offsets_pass_32_bits():
    import torch
    n, d, vr, vp, ld = 1100, 64, 1090, 1152, 1 << 21
    say(f"case: {n} rows {ld} elements apart")
    p = Problem(23, n, d, vr, vp)
    want = run_all(p)
    a, kw = p.args()
    far = [torch.empty((k, ld), dtype=t, device="cuda:0")[:, ld - d:] for k, t in
           ((n, torch.bfloat16), (vr, torch.bfloat16), (n, torch.float32), (vr, torch.float32))]
    far[0].copy_(p.h)
    far[1].copy_(p.w)
    gh, gw = rlk.linear_logp_backward(far[0], far[1], *a[2:], **kw, grad_hidden=far[2], grad_weight=far[3])
    assert np.array_equal(bits(gh.to(torch.bfloat16)), bits(want[0]))
    assert np.array_equal(bits(gw.to(torch.bfloat16)), bits(want[1]))


@pytest.mark.parametrize("vr,vp", [(2000, 2048), (500, 2048), (1000, 1088), (60, 64)])
def test_vocabulary_parallel_parts_give_the_bytes_of_the_whole(vr, vp):
    import torch
    say(f"case: ranks of {vr} of {vp}")
    p = Problem(14, 50, 192, vr, vp)
    gh, gw = run_all(p)
    for groups in (1, 2, 4, 8):
        cols = vp // groups
        parts, rows = [], []
        for rank in range(groups):
            a, kw = p.args()
            lo, hi = min(vr, rank * cols), min(vr, (rank + 1) * cols)
            w = p.w[lo:hi]
            part, wg = rlk.linear_logp_backward(a[0], w, *a[2:], **kw, vocab_real=vr, rank=rank, groups=groups,
                                                grad_hidden=torch.empty((p.n, p.d), device=w.device))
            parts.append(part)
            rows.append(wg)
        got = rlk.linear_logp_backward_merge(torch.stack(parts))
        assert np.array_equal(bits(got), bits(gh)), f"grad_hidden at {groups} ranks"
        assert np.array_equal(bits(torch.cat(rows)), bits(gw)), f"grad_weight at {groups} ranks"
        wide = torch.full((p.n, p.d + 8), 7.0, device="cuda:0")
        rlk.linear_logp_backward_merge(torch.stack(parts), out=wide[:, :p.d])
        assert np.array_equal(bits(wide[:, :p.d].to(torch.bfloat16)), bits(gh)) and bool((wide[:, p.d:] == 7.0).all())


def test_agrees_with_the_gradient_of_kept_logits():
    """The same G as rlk_logp_backward on rlk_linear's logits, to the byte: with an
    identity as hidden states grad_weight is G^T, rounded once more to itself."""
    import torch
    say("case: G against logp_backward")
    n = 256
    p = Problem(15, n, n, 3000, 3008, top_p=0.9)
    eye = torch.eye(n, dtype=torch.bfloat16, device="cuda:0")
    p.h = eye * 4
    p.forward()
    _, gw = run_all(p, "both")
    G = rlk.logp_backward(p.logits, p.t, p.tg, vocab_real=p.vr, ref_logp=p.ref, lse=p.lse, grad_ref=f32(p.g_ref),
                          policy_logp=p.pol, support_state=p.state, grad_policy=f32(p.g_pol))
    want = (G[:, :p.vr].float() * 4).to(torch.bfloat16).T
    assert np.array_equal(bits(gw) & 0x7FFF, bits(want) & 0x7FFF)  # -0 becomes 0 in a sum
    assert bool((gw == want).all())


def test_against_differences_of_the_forward():
    """The derivative along a random direction of the projection and of the hidden
    states, from the oracle's logprobs with unrounded logits, against the
    gradients' inner product with it. Errors: BF16 logits (2^-8 of about 10, a
    few per cent of a weight) and the difference's own 1e-6."""
    say("case: differences")
    p = Problem(16, 6, 128, 200, 256, temps=(1.0,), lean=1.0)
    gh, gw = run_all(p)
    h, w = LIN.bf16_to_f64(p.hb), LIN.bf16_to_f64(p.wb)
    g = p.g_ref.astype(np.float64)

    def loss(h, w):
        x = h @ w.T
        m = x.max(1, keepdims=True)
        lse = m[:, 0] + np.log(np.exp(x - m).sum(1))
        return float((g * (x[np.arange(p.n), p.target] - lse)).sum())

    rng = np.random.default_rng(2)
    for _ in range(4):
        dh, dw = rng.normal(0, 1, h.shape), rng.normal(0, 1, w.shape)
        got_h = float((to_host(gh.double()) * dh).sum())
        got_w = float((to_host(gw.double()) * dw).sum())
        e = 1e-5
        want_h = (loss(h + e * dh, w) - loss(h - e * dh, w)) / (2 * e)
        want_w = (loss(h, w + e * dw) - loss(h, w - e * dw)) / (2 * e)
        # G moves by at most 2^-8 |x| <= 0.06 of each p beside its own rounding; the
        # errors add as the square root of their number: 0.06 of the gradient's norm
        # (a direction's standard deviation) three times over
        assert abs(got_h - want_h) <= 0.18 * np.linalg.norm(to_host(gh.double())) + 1e-4
        assert abs(got_w - want_w) <= 0.18 * np.linalg.norm(to_host(gw.double())) + 1e-4


def test_another_stream_and_two_at_once():
    import torch
    say("case: side streams")
    ps = [Problem(20 + k, 130, 256, 1500, 1536) for k in range(2)]
    want = [run_all(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for _ in range(3):
        got = [run_all(p, stream=s) for p, s in zip(ps, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert np.array_equal(bits(a[0]), bits(b[0])) and np.array_equal(bits(a[1]), bits(b[1]))


def test_captured_and_replayed_with_other_rows_masked():
    """Two graphs with a workspace each; every replay against the eager result."""
    import torch
    say("case: graphs")
    p = Problem(22, 150, 192, 1000, 1024)
    a, kw = p.args()
    outs, graphs = [], []
    need = rlk.linear_logp_backward_workspace_bytes(p.n, p.d, p.vp, p.vr)
    for _ in range(2):
        gh, gw = torch.empty((p.n, p.d), dtype=torch.bfloat16, device="cuda:0"), torch.zeros((p.vr, p.d), device="cuda:0")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda:0")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                rlk.linear_logp_backward(*a, **kw, grad_hidden=gh, grad_weight=gw, workspace=ws)
        outs.append((gh, gw))
        graphs.append(g)
    rng = np.random.default_rng(4)
    for step in range(4):
        kw["grad_ref"].copy_(f32(p.g_ref * (rng.random(p.n) < 0.7) if step else np.zeros(p.n)))
        want = rlk.linear_logp_backward(*a, **kw, grad_weight=torch.empty((p.vr, p.d), device="cuda:0"))
        for g, (gh, gw) in zip(graphs, outs):
            gh.fill_(9)
            gw.fill_(9)
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(bits(gh), bits(want[0])) and np.array_equal(bits(gw), bits(want[1])), f"replay {step}"
