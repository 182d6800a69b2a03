"""GPU parity of the verification of drafted tokens against the float64 oracle
(oracle/draft.py), on statistics that logp_nucleus itself produced.

Tokens and accepted counts must be equal: both sides work in float64 from the
same float32 statistics, so a drawn token can differ only where the random
number lies within the float64 sums' rounding of a column's border. With up to
152,000 terms of at most 1, each exponential off by a few 2^-52 and each sum by
2^-53, that is below 1e-10 of the whole weight; every comparison checks that
the drawn tokens' borders are further away than that. The logprobs are one
float32 rounding of a difference: 2^-24 of the value.
"""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import draft as OD

from gpu_util import say, to_host

pytestmark = pytest.mark.gpu

BORDER = 1e-10


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to("cuda:0")


def logits_of(bits, stride=None):
    import torch
    n, v = bits.shape
    buf = np.full((n, stride or v), 0x7FC0, dtype=np.uint16)
    buf[:, :v] = bits
    return torch.from_numpy(buf.view(np.int16)).to("cuda:0").view(torch.bfloat16)


class Batch:
    """A batch of sequences with drafted tokens; `score` lets logp_nucleus fill in the statistics."""

    def __init__(self, rng, counts, vr, vp, temps=(1.0,), top_p=1.0, top_k=-1, drafter="sampled", noise=0.5, sigma=2.5,
                 stride=None, spare=0):
        self.vr, self.vp = vr, vp
        n = len(counts)
        self.start = np.concatenate(([0], np.cumsum(counts))).astype(np.int64)
        nd = int(self.start[-1])
        rows = nd + n + spare
        seq = np.repeat(np.arange(n), counts)
        self.row = np.arange(nd) + seq
        x = rng.normal(0, sigma, (rows, vr))
        self.bits = self.pad(x)
        self.q_bits = self.pad(x[self.row] + noise * rng.normal(0, 1, (nd, vr)))
        t_seq = rng.choice(np.array(temps, np.float32), n)
        self.t = np.concatenate((np.repeat(t_seq, np.asarray(counts) + 1), np.ones(spare, np.float32))).astype(np.float32)
        self.tq = t_seq[seq].astype(np.float32)
        self.top_p, self.top_k = top_p, top_k
        self.token = np.zeros(nd, np.int64)
        for i in range(nd):   # what a drafter would draw: from its softmax, or its maximum
            z = OD.decode_bf16(self.q_bits[i, :vr])
            if self.tq[i] == 0:
                self.token[i] = int(np.argmax(z))
            else:
                g = -np.log(-np.log(rng.random(vr) * (1 - 2e-16) + 1e-16))
                order = np.argsort(-z, kind="stable")[:max(1, vr // 3)] if top_p < 1 or top_k != -1 else np.arange(vr)
                self.token[i] = int(order[np.argmax(z[order] / self.tq[i] + g[order])])
        self.accept_u = rng.random(nd)
        self.sample_u = rng.random(n)
        self.drafter = drafter
        self.stride = stride
        self.scored = False

    def pad(self, x):
        b = np.full((len(x), self.vp), 0xFF80, np.uint16)
        b[:, :self.vr] = datagen.f32_to_bf16_bits(np.asarray(x, np.float32))
        return b

    def score(self):
        import torch

        def forward(bits, t, token):
            lg = logits_of(bits, self.stride)
            n = len(t)
            pol, ref, lse, state = rlk.logp_nucleus(lg, dev(t), self.top_p, self.top_k, dev(token),
                                                    vocab_real=self.vr, vocab_padded=self.vp, return_state=True)
            torch.cuda.synchronize()
            part, thr, status = (to_host(f.contiguous()) for f in rlk.support_state_fields(state))
            rows = OD.Rows(bits, t, to_host(pol), part, thr, status, to_host(ref), to_host(lse))
            assert len(part) == n
            return lg, (pol, ref, lse, state), rows

        target = np.zeros(len(self.t), np.int64)
        target[self.row] = self.token
        self.lg, self.stats, self.rows = forward(self.bits, self.t, target)
        self.qlg = None
        if self.drafter == "sampled" and len(self.token):
            self.qlg, self.qstats, self.q_rows = forward(self.q_bits, self.tq, self.token)
        self.scored = True
        return self

    def call(self, **kw):
        import torch
        pol, ref, lse, state = self.stats
        more = {}
        if self.qlg is not None:
            more = dict(draft_logits=self.qlg, draft_temperature=dev(self.tq), draft_policy_logp=self.qstats[0],
                        draft_support_state=self.qstats[3])
        got = rlk.draft_verify(self.lg, dev(self.token), dev(self.start), dev(self.accept_u), dev(self.sample_u),
                               temperature=dev(self.t), policy_logp=pol, ref_logp=ref, lse=lse, support_state=state,
                               vocab_real=self.vr, vocab_padded=self.vp, **more, **kw)
        torch.cuda.synchronize()
        return [to_host(g) for g in got]

    def want(self):
        return OD.verify(self.rows, self.q_rows if self.qlg is not None else None, self.vr, self.start, self.token,
                         self.accept_u, self.sample_u)

    def check(self, used=None, **kw):
        got, want = self.call(**kw), self.want()
        used = used if used is not None else int(self.start[-1]) + len(self.start) - 1
        assert want[4].min() > BORDER, "a random number lies on a border: choose another seed"
        assert np.array_equal(got[1], want[1]), "accepted counts"
        assert np.array_equal(got[0][:used], want[0][:used]), "tokens"
        for g, w, what in ((got[2], want[2], "policy"), (got[3], want[3], "reference")):
            g, w = g[:used].astype(np.float64), w[:used]
            assert np.array_equal(np.isnan(g), np.isnan(w)), what
            fine = ~np.isnan(w)
            assert (np.abs(g[fine] - w[fine]) <= 2.0 ** -24 * np.abs(w[fine]) * (1 + 1e-6)).all(), what
        return got


CASES = [
    # counts, vr, vp, temps, top_p, top_k, drafter
    ([4], 151936, 152576, (1.0,), 1.0, -1, "sampled"),
    ([0, 1, 2, 3, 4, 5], 151936, 152576, (0.7,), 0.95, -1, "sampled"),
    ([3] * 40, 5000, 5056, (0.7, 1.0, 1.3, 0.0), 1.0, -1, "sampled"),
    ([3] * 40, 5000, 5056, (0.7, 1.0, 1.3, 0.0), 1.0, -1, "point"),
    ([2] * 60, 2047, 2048, (1.0,), 0.9, -1, "sampled"),
    ([2] * 60, 2048, 2112, (1.0,), 1.0, 50, "sampled"),
    ([2] * 60, 2049, 2112, (2.0,), 0.5, 300, "point"),
    ([0] * 50, 4099, 4160, (0.7, 0.0, 5.0), 0.99, -1, "sampled"),
    ([1] * 64, 7, 64, (1.0, 0.3), 1.0, -1, "sampled"),
    ([1] * 64, 1, 64, (1.0, 0.0), 1.0, -1, "sampled"),
    ([0, 7, 0, 0, 63, 64, 65, 200, 1], 700, 704, (1.0,), 1.0, -1, "sampled"),
    ([1] * 500, 130000, 130048, (1.0,), 1.0, -1, "point"),
    # more pieces of 512 columns than a workgroup keeps: few and many sequences
    ([2, 0, 1], 300001, 300032, (0.9,), 1.0, -1, "sampled"),
    ([1] * 140, 262145, 262208, (1.0, 0.0), 0.98, -1, "sampled"),
    # around the numbers of sequences at which the work is shared out in another way
    ([1] * 8, 151936, 152576, (0.8, 0.0), 1.0, -1, "sampled"),
    ([1] * 14, 151936, 152576, (0.8, 0.0), 1.0, -1, "sampled"),
    ([2] * 128, 9000, 9024, (0.7,), 0.9, -1, "sampled"),
    ([2] * 129, 9000, 9024, (0.7, 1.3), 1.0, -1, "sampled"),
    ([1] * 257, 9000, 9024, (0.7, 1.3), 1.0, 400, "sampled"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_verify_matches_the_oracle(case):
    counts, vr, vp, temps, top_p, top_k, drafter = CASES[case]
    say(f"case: verify {len(counts)} sequences, {sum(counts)} drafted, vocab {vr}, T {temps}, top-p {top_p}, {drafter}")
    rng = np.random.default_rng(100 + case)
    n_rows = sum(counts) + len(counts)
    # long drafts need likely tokens: little noise
    b = Batch(rng, counts, vr, vp, temps, top_p, top_k, drafter, noise=0.02 if max(counts) > 8 else 0.5,
              stride=vp + 8 * (case % 3))
    got = b.score().check()
    if max(counts) > 8:
        assert got[1].max() > 64    # accepted tokens beyond the first 64
    assert n_rows == len(got[0])


def test_every_column_can_be_drawn():
    """Equal logits: column j of 4099 is drawn by the random number (j + 1/2) / 4099."""
    say("case: each of 4099 columns drawn")
    v, vp = 4099, 4160
    b = Batch(np.random.default_rng(1), [0] * v, v, vp)
    b.bits[:, :v] = 0x3F80
    b.sample_u = (np.arange(v) + 0.5) / v
    got = b.score().check()
    assert np.array_equal(got[0], np.arange(v))


def test_ends_of_the_unit_interval():
    """sample_u 0 takes the first column of any weight, the largest number
    below 1 the last; accept_u 0 accepts any token that has policy mass."""
    say("case: random numbers at the ends")
    rng = np.random.default_rng(2)
    vr, vp = 3000, 3008
    b = Batch(rng, [1] * 64, vr, vp, (1.0,), 0.6, -1, "sampled")
    b.sample_u = np.where(np.arange(64) % 2 == 0, 0.0, 1 - 2.0 ** -53)
    b.accept_u = np.where(np.arange(64) % 4 < 2, 0.0, 1 - 2.0 ** -53)
    b.score()
    got, want = b.call(), b.want()
    assert np.array_equal(got[1], want[1])
    n_refused = 0
    for s in range(64):
        k = int(got[1][s])
        row = 2 * s + k
        r = OD.distribution(b.rows, row, vr)
        if k == 0:
            r = np.maximum(r - OD.distribution(b.q_rows, s, vr), 0)
            n_refused += 1
        weighted = np.flatnonzero(r > 0)
        if not weighted.size:   # a token outside both policies, which are the same point mass: nothing is left
            assert got[0][row] == -1 and np.isnan(got[2][row])
            continue
        assert got[0][row] == (weighted[0] if s % 2 == 0 else weighted[-1])
        if s % 4 < 2:
            assert k == (1 if b.rows.policy[2 * s] > -np.inf else 0)
    assert 0 < n_refused < 64


def test_greedy_rows_and_ties():
    """Greedy targets: the lowest column of the maximum, -0 equal to 0, across
    chunks and at both ends; greedy drafts are point masses."""
    say("case: greedy rows")
    vr, vp = 6001, 6016
    b = Batch(np.random.default_rng(3), [1] * 12, vr, vp, (0.0,))
    where = [[0, 6000], [6000], [2047, 2048], [2048, 4096], [5, 4097], [4095, 4096, 6000], [0], [1, 2], [511, 512], [8, 9],
             [4096], [3000, 5999]]
    b.bits[:, :vr] = 0xC000                     # -2
    for s, cols in enumerate(where):
        for row in (2 * s, 2 * s + 1):
            b.bits[row, cols] = 0x8000 if s % 2 else 0x3F80
            if s % 2:
                b.bits[row, cols[-1]] = 0x0000
    b.token[:] = [w[0] if i % 3 else w[-1] for i, w in enumerate(where)]
    got = b.score().check()
    for s, cols in enumerate(where):
        assert got[0][2 * s] == cols[0]
        assert got[1][s] == (1 if b.token[s] == cols[0] else 0)
        assert got[2][2 * s] == 0.0 and got[3][2 * s] == 0.0


def test_equal_rows_accept_and_rounded_statistics_fall_back():
    say("case: the drafter's rows are the target's")
    b = Batch(np.random.default_rng(4), [2] * 20, 900, 960, (0.9,), 0.9, -1, "sampled")
    b.q_bits = b.bits[b.row].copy()
    b.accept_u[:] = 1 - 2.0 ** -53
    # tokens of the support: the maximum and a copy of it
    b.token[:] = [int(np.argmax(OD.decode_bf16(q[:900]))) for q in b.q_bits]
    got = b.score().check()
    assert (got[1] == 2).all()
    # the same with the draft's logprob one step higher: refused, nothing left over, the drafted token stays
    pol = b.qstats[0]
    pol.copy_(pol + 1e-5)
    b.q_rows = b.q_rows._replace(policy=to_host(pol))
    got = b.check()
    assert (got[1] == 0).all() and np.array_equal(got[0][0::3], b.token[0::2])


def test_what_cannot_be_served():
    """NaN and infinite logits, an invalid top-k, drafted tokens and random
    numbers out of range end a sequence with token -1 and NaN; offsets out of
    order leave everything but accepted_out = -1; the other sequences and the
    rows behind the last one are untouched."""
    import torch
    say("case: invalid rows, tokens, numbers, offsets")
    vr, vp, n = 2100, 2112, 16
    b = Batch(np.random.default_rng(5), [2] * n, vr, vp, (1.0,), 0.9, -1, "sampled", spare=3)
    b.accept_u[:] = 0.0
    b.token[:] = [int(np.argmax(OD.decode_bf16(q[:vr]))) for q in b.q_bits]
    b.bits[3 * 1, 700] = 0x7FC0              # sequence 1: NaN in its first row
    b.bits[3 * 2 + 2, 5] = 0x7F80            # 2: +inf in the row behind its drafts
    b.q_bits[2 * 3 + 1, 9] = 0xFFC0          # 3: NaN in the draft's second row
    b.token[2 * 4] = vr                      # 4, 5: tokens out of range
    b.token[2 * 5 + 1] = -1
    b.accept_u[2 * 6] = 1.0                  # 6, 7, 8: numbers
    b.accept_u[2 * 7 + 1] = np.nan
    b.accept_u[2 * 8] = -0.25
    b.sample_u[9], b.sample_u[10], b.sample_u[11] = 1.0, np.nan, -1e-300
    b.t[3 * 12:3 * 13] = np.nan              # 12, 13: temperatures
    b.t[3 * 13 + 2] = -1.0
    b.bits[3 * 14 + 2, :vr] = 0xFF80         # 14: no logit above -inf
    b.score()
    outs = dict(token_out=torch.full((len(b.t),), 77, dtype=torch.int64, device="cuda:0"),
                accepted_out=torch.full((n,), 77, dtype=torch.int32, device="cuda:0"),
                policy_out=torch.full((len(b.t),), 77.0, device="cuda:0"),
                ref_out=torch.full((len(b.t),), 77.0, device="cuda:0"))
    got = b.check(**outs)
    assert [got[1][s] for s in (1, 2, 3, 4, 5, 6, 7, 8, 12, 13, 14)] == [0, 2, 1, 0, 1, 0, 1, 0, 0, 2, 2]
    for s in (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14):
        at = 3 * s + got[1][s]
        assert got[0][at] == -1 and np.isnan(got[2][at]) and np.isnan(got[3][at])
    for s in (0, 15):
        assert (got[0][3 * s:3 * s + got[1][s] + 1] >= 0).all()
    for g in (got[0], got[2], got[3]):
        assert (g[3 * n:] == 77).all()
    # offsets: out of order, below 0, behind the last drafted token
    b.start[4], b.start[9] = 11, 2 * n + 1
    b.start[0] = -1
    for t in outs.values():
        t.fill_(77)
    got = b.call(**outs)
    want = b.want()
    assert np.array_equal(got[1], want[1]) and (want[1][[0, 4, 8, 9]] == -1).all()
    assert (got[0][0:2] == 77).all()


def test_values_outside_the_table():
    """Rows of many columns, so that weights come from the table, with zeros, -0,
    tiny, huge and -inf values among them, and a support of exactly those."""
    say("case: zeros, tiny and huge logits")
    rng = np.random.default_rng(14)
    vr, vp, n = 40000, 40064, 140
    b = Batch(rng, [1] * n, vr, vp, (1.0, 7.0), 1.0, -1, "sampled")
    odd = np.array([0.0, -0.0, 1e-20, -1e-20, 2.0 ** -13, -(2.0 ** -13), 63.75, 64.0, -64.0, -700.0, -1e4, -3e38, -np.inf])
    for bits in (b.bits, b.q_bits):
        where = rng.random((len(bits), vr)) < 0.3
        values = rng.choice(odd, (len(bits), vr))
        values[values > 60] = np.where(rng.random((values > 60).sum()) < 0.001, values[values > 60], 0.0)
        bits[:, :vr][where] = datagen.f32_to_bf16_bits(values.astype(np.float32))[where]
    got = b.score().check()
    assert (got[0][:2 * n:2] >= 0).all()


def test_unusable_statistics_of_the_draft():
    """A draft row whose record or temperature is not a number ends its
    sequence there; it is never taken for a drafter that gives nothing."""
    say("case: NaN in the draft's statistics")
    import torch
    b = Batch(np.random.default_rng(15), [1] * 4, 3000, 3008, (1.0,), 1.0, -1, "sampled").score()
    b.accept_u[:] = 1 - 2.0 ** -53
    b.qstats[3].view(torch.float32)[0, 0] = float("nan")   # lse_support, status left at 1
    b.tq[1] = np.nan
    b.tq[2] = -1.0
    got = b.call()
    assert got[1][:3].tolist() == [0, 0, 0]
    assert (got[0][[0, 2, 4]] == -1).all() and np.isnan(got[2][[0, 2, 4]]).all()


def test_offsets_past_31_bits():
    """Sequences at the end of 14,100 rows of 152,576 columns (more than 2^31
    elements): as in a call on those rows alone."""
    import torch
    say("case: rows past 2^31 elements")
    b = Batch(np.random.default_rng(16), [2, 0, 3, 1], 151936, 152576, (0.8,), 1.0, -1, "sampled").score()
    want = b.check()
    nd, n, big = len(b.token), 4, 14100
    rows = big + nd + n

    def tail(t, total):
        shape = (total,) + tuple(t.shape[1:])
        out = torch.zeros(shape, dtype=t.dtype, device="cuda:0")
        out[total - t.shape[0]:] = t
        return out

    pol, ref, lse, state = b.stats
    got = rlk.draft_verify(
        tail(b.lg, rows), tail(dev(b.token), big + nd), dev(b.start) + big, tail(dev(b.accept_u), big + nd), dev(b.sample_u),
        temperature=tail(dev(b.t), rows), policy_logp=tail(pol, rows), ref_logp=tail(ref, rows), lse=tail(lse, rows),
        support_state=tail(state, rows), vocab_real=b.vr, vocab_padded=b.vp, draft_logits=tail(b.qlg, big + nd),
        draft_temperature=tail(dev(b.tq), big + nd), draft_policy_logp=tail(b.qstats[0], big + nd),
        draft_support_state=tail(b.qstats[3], big + nd))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert to_host(g[g.shape[0] - len(w):]).tobytes() == w.tobytes()
    assert (to_host(got[0][:big]) == -1).all()


def test_inf_rows_in_masked_places():
    """-inf logits inside the vocabulary, columns behind it that hold NaN, and
    values below the support's threshold never weigh anything."""
    say("case: -inf logits, NaN in the pad columns")
    b = Batch(np.random.default_rng(6), [1] * 32, 2500, 2560, (0.8,), 0.8, -1, "sampled")
    rng = np.random.default_rng(7)
    for bits in (b.bits, b.q_bits):
        mask = rng.random((len(bits), 2500)) < 0.7
        mask[:, ::100] = False
        bits[:, :2500][mask] = 0xFF80
        bits[:, 2500:] = 0x7FC0
    b.token[:] = [int(np.argmax(OD.decode_bf16(q[:2500]))) for q in b.q_bits]
    got = b.score().check()
    for row, tok in enumerate(got[0]):
        assert tok < 0 or b.bits[row, tok] != 0xFF80


def test_a_sequence_does_not_depend_on_the_batch():
    say("case: one sequence in many batches")
    rng = np.random.default_rng(8)
    counts = [int(c) for c in rng.integers(0, 5, 600)]
    b = Batch(rng, counts, 9000, 9024, (0.7, 1.0, 0.0), 0.97, -1, "sampled").score()
    whole = b.check()
    import torch
    pol, ref, lse, state = b.stats
    for lo, hi in ((0, 1), (5, 6), (599, 600), (10, 74), (100, 400), (0, 300)):
        d0, d1 = b.start[lo], b.start[hi]
        r0, r1 = d0 + lo, d1 + hi
        got = rlk.draft_verify(b.lg[r0:r1], dev(b.token[d0:d1]), dev(b.start[lo:hi + 1] - d0), dev(b.accept_u[d0:d1]),
                               dev(b.sample_u[lo:hi]), temperature=dev(b.t[r0:r1]), policy_logp=pol[r0:r1],
                               ref_logp=ref[r0:r1], lse=lse[r0:r1], support_state=state[r0:r1], vocab_real=b.vr,
                               vocab_padded=b.vp, draft_logits=b.qlg[d0:d1], draft_temperature=dev(b.tq[d0:d1]),
                               draft_policy_logp=b.qstats[0][d0:d1], draft_support_state=b.qstats[3][d0:d1])
        torch.cuda.synchronize()
        for g, w, at in zip(got, whole, (slice(r0, r1), slice(lo, hi), slice(r0, r1), slice(r0, r1))):
            assert to_host(g).tobytes() == w[at].tobytes(), (lo, hi)


def test_calls_on_two_streams_at_once():
    """The same call on two side streams that are not waited for, with outputs
    and workspaces of its own making, many times: as on the main stream."""
    import torch
    say("case: two streams at once")
    b = Batch(np.random.default_rng(13), [3] * 50, 20000, 20032, (0.7, 1.0, 0.0), 0.97, -1, "sampled").score()
    want = [w.tobytes() for w in b.check()]
    pol, ref, lse, state = b.stats
    args = (b.lg, dev(b.token), dev(b.start), dev(b.accept_u), dev(b.sample_u))
    kw = dict(temperature=dev(b.t), policy_logp=pol, ref_logp=ref, lse=lse, support_state=state, vocab_real=b.vr,
              vocab_padded=b.vp, draft_logits=b.qlg, draft_temperature=dev(b.tq), draft_policy_logp=b.qstats[0],
              draft_support_state=b.qstats[3])
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [rlk.draft_verify(*args, **kw, stream=sides[i % 2]) for i in range(20)]
    noise = [torch.full((len(b.t),), 9.0, device="cuda:0") for _ in range(40)]   # memory that the side streams' may not be
    torch.cuda.synchronize()
    for g in got:
        assert [to_host(t).tobytes() for t in g] == want
    assert all((t == 9.0).all() for t in noise)


def test_graph_replays_with_other_lengths():
    """Two captured calls, each with a workspace of its own, replayed with new
    offsets, tokens and numbers, eager calls and poisoned outputs between."""
    import torch
    say("case: two captured calls")
    rng = np.random.default_rng(9)
    vr, vp, kept = 5000, 5056, []
    for n, most in ((6, 4), (90, 2)):
        nd = n * most
        b = Batch(rng, [most] * n, vr, vp, (1.0,), 0.95, -1, "sampled").score()
        start, token, au, su = dev(b.start), dev(b.token), dev(b.accept_u), dev(b.sample_u)
        t, tq = dev(b.t), dev(b.tq)
        out = dict(token_out=torch.zeros(nd + n, dtype=torch.int64, device="cuda:0"),
                   accepted_out=torch.zeros(n, dtype=torch.int32, device="cuda:0"),
                   policy_out=torch.zeros(nd + n, device="cuda:0"), ref_out=torch.zeros(nd + n, device="cuda:0"))
        ws = torch.zeros(rlk.draft_workspace_bytes(n, vp, vr), dtype=torch.uint8, device="cuda:0")
        pol, ref, lse, state = b.stats

        def call(out=out, ws=ws, b=b, start=start, token=token, au=au, su=su, t=t, tq=tq, pol=pol, ref=ref, lse=lse,
                 state=state):
            return rlk.draft_verify(b.lg, token, start, au, su, temperature=t, policy_logp=pol, ref_logp=ref, lse=lse,
                                    support_state=state, vocab_real=vr, vocab_padded=vp, draft_logits=b.qlg,
                                    draft_temperature=tq, draft_policy_logp=b.qstats[0], draft_support_state=b.qstats[3],
                                    workspace=ws, **out)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        kept.append((n, most, start, au, su, out, ws, call, g))
    for again in range(4):
        for n, most, start, au, su, out, ws, call, g in kept:
            # other lengths within the captured capacity: the rows then belong to other sequences
            counts = rng.integers(0, most + 1, n) if again else np.full(n, most)
            start.copy_(dev(np.concatenate(([0], np.cumsum(counts))).astype(np.int64)))
            au.copy_(dev(rng.random(n * most)))
            su.copy_(dev(rng.random(n)))
            for v in out.values():
                v.fill_(9)
            call()
            torch.cuda.synchronize()
            want = [to_host(v).tobytes() for v in out.values()]
            for v in out.values():
                v.fill_(9)
            ws.fill_(0x5C)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert [to_host(v).tobytes() for v in out.values()] == want, (again, n)


def test_emitted_tokens_follow_the_targets_policy():
    """40,000 sequences of one drafted token on the same pair of rows, random
    numbers from a seeded generator: the first emitted tokens' counts against
    the target's policy, each within 5 standard deviations."""
    say("case: distribution of 40000 emitted tokens")
    rng = np.random.default_rng(10)
    n, vr, vp = 40000, 12, 64
    b = Batch(rng, [1] * n, vr, vp)
    b.bits[:] = b.bits[:1]
    b.q_bits[:] = b.pad(rng.normal(0, 2.0, (1, vr)))
    q = np.exp(OD.decode_bf16(b.q_bits[0, :vr]))
    b.token = rng.choice(vr, n, p=q / q.sum()).astype(np.int64)
    got = b.score().call()
    first = got[0][0::2]
    p = OD.distribution(b.rows, 0, vr)
    p = p / p.sum()
    off = np.abs(np.bincount(first, minlength=vr) - n * p)
    assert (off <= 5 * np.sqrt(n * p * (1 - p)) + 1).all()
    assert 0.05 * n < got[1].sum() < 0.95 * n


def test_drafting_with_the_4_bit_head_and_verifying_with_the_bf16_head():
    """The operators as they are used together: the head quantised once; three
    tokens drafted from its logits, one call of the sampler each; the BF16
    head's logits of all four places; their statistics; the verification, and
    the emitted tokens' logprobs against logp_nucleus on those tokens."""
    import torch
    say("case: draft with the 4-bit head, verify with the BF16 head")
    rng = np.random.default_rng(11)
    n, most, d, vr, vp = 24, 3, 512, 6000, 6016
    w = dev(datagen.f32_to_bf16_bits((rng.normal(0, 2.5 / np.sqrt(d), (vr, d))).astype(np.float32)).view(np.int16)).view(torch.bfloat16)
    wc, ws = rlk.mx4_quantize(w)
    hidden = dev(datagen.f32_to_bf16_bits(rng.normal(0, 1, (n, most + 1, d)).astype(np.float32)).view(np.int16)).view(torch.bfloat16)
    t, top_p, top_k = 0.9, 0.98, -1
    one = torch.arange(n + 1, device="cuda:0") * 0
    drafted, drafts = [], []
    zero, none = torch.zeros(n, dtype=torch.int64, device="cuda:0"), torch.zeros(0, dtype=torch.int64, device="cuda:0")
    for k in range(most):   # a drafter's step: logits of 4-bit operands, the support, a token of it
        lg = rlk.mx4_linear(hidden[:, k], wc, ws, vocab_real=vr, vocab_padded=vp)
        pol, ref, lse, state = rlk.logp_nucleus(lg, t, top_p, top_k, zero, vocab_real=vr, return_state=True)
        tok, acc, qpol, _ = rlk.draft_verify(lg, none, one, none.double(), dev(rng.random(n)), temperature=t, policy_logp=pol,
                                             ref_logp=ref, lse=lse, support_state=state, vocab_real=vr)
        assert (to_host(acc) == 0).all()
        again, _, _, state = rlk.logp_nucleus(lg, t, top_p, top_k, tok, vocab_real=vr, return_state=True)
        assert (torch.abs(again - qpol) <= 2.0 ** -22 * torch.abs(again).clamp(min=1)).all()   # one float32 step of lse_support
        drafted.append(tok)
        drafts.append((lg, qpol, state))
    token = torch.stack(drafted, 1).reshape(-1).contiguous()
    q_logits = torch.stack([x[0] for x in drafts], 1).reshape(n * most, vp)
    q_pol = torch.stack([x[1] for x in drafts], 1).reshape(-1).contiguous()
    q_state = torch.stack([x[2] for x in drafts], 1).reshape(n * most, 4).contiguous()
    start = torch.arange(n + 1, device="cuda:0") * most
    logits = rlk.linear(hidden.reshape(n * (most + 1), d), w, vocab_padded=vp)
    target = torch.zeros((n, most + 1), dtype=torch.int64, device="cuda:0")
    target[:, :most] = token.view(n, most)
    pol, ref, lse, state = rlk.logp_nucleus(logits, t, top_p, top_k, target.view(-1), vocab_real=vr, return_state=True)
    accept_u, sample_u = rng.random(n * most), rng.random(n)
    out, acc, opol, oref = rlk.draft_verify(
        logits, token, start, dev(accept_u), dev(sample_u), temperature=t, policy_logp=pol, ref_logp=ref, lse=lse,
        support_state=state, vocab_real=vr, draft_logits=q_logits, draft_temperature=t, draft_policy_logp=q_pol,
        draft_support_state=q_state)
    torch.cuda.synchronize()

    def rows(lg, p, s, r=None, e=None):
        part, thr, status = (to_host(f.contiguous()) for f in rlk.support_state_fields(s))
        bits = to_host(lg.view(torch.int16)).view(np.uint16)
        return OD.Rows(bits, np.full(len(bits), t, np.float32), to_host(p), part, thr, status,
                       to_host(r) if r is not None else None, to_host(e) if e is not None else None)

    want = OD.verify(rows(logits, pol, state, ref, lse), rows(q_logits, q_pol, q_state), vr, to_host(start), to_host(token),
                     accept_u, sample_u)
    assert want[4].min() > BORDER
    assert np.array_equal(to_host(out), want[0]) and np.array_equal(to_host(acc), want[1])
    assert 0 < to_host(acc).sum() < n * most      # some accepted, some refused
    # what the trainer would compute for the emitted tokens: within a float32 step or two of the statistics
    emitted = out >= 0
    pol2, ref2 = rlk.logp_nucleus(logits, t, top_p, top_k, out.clamp(min=0), vocab_real=vr)
    for a, c in ((opol, pol2), (oref, ref2)):
        a, c = to_host(a[emitted]).astype(np.float64), to_host(c[emitted]).astype(np.float64)
        assert (np.abs(a - c) <= 2.0 ** -22 * np.maximum(np.abs(c), 16)).all()


def test_refusals_on_the_device():
    import torch
    b = Batch(np.random.default_rng(12), [1] * 4, 100, 128).score()
    pol, ref, lse, state = b.stats
    base = dict(logits=b.lg, draft_token=dev(b.token), draft_start=dev(b.start), accept_u=dev(b.accept_u),
                sample_u=dev(b.sample_u), temperature=dev(b.t), policy_logp=pol, ref_logp=ref, lse=lse, support_state=state,
                vocab_real=100, vocab_padded=128)
    rlk.draft_verify(**base)
    for kw in (dict(logits=b.lg[:7]), dict(draft_token=dev(b.token.astype(np.int32))), dict(draft_start=dev(b.start)[:0]),
               dict(accept_u=dev(b.accept_u).float()), dict(accept_u=dev(b.accept_u)[:3]), dict(sample_u=dev(b.sample_u)[:3]),
               dict(temperature=dev(b.t)[:5]), dict(policy_logp=None), dict(ref_logp=ref[:3]), dict(lse=lse.double()),
               dict(support_state=state[:, :3]), dict(vocab_padded=192), dict(draft_logits=b.qlg[:3]),
               dict(draft_logits=b.qlg), dict(token_out=torch.empty(3, dtype=torch.int64, device="cuda:0")),
               dict(accepted_out=torch.empty(4, dtype=torch.int64, device="cuda:0")),
               dict(policy_out=torch.empty(8, dtype=torch.float64, device="cuda:0")),
               dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda:0"))):
        with pytest.raises(ValueError):
            rlk.draft_verify(**{**base, **kw})
    with pytest.raises(rlk.RlkError):
        rlk.draft_verify(**{**base, "vocab_real": 129})
    with pytest.raises(rlk.RlkError):
        rlk.draft_verify(**{**base, "vocab_real": 0})
