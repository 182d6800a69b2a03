"""GPU parity of the verification on rows that cannot be served, against the
float64 oracle (oracle/draft.py) on the same statistics. Tokens and counts are
equal, logprobs those of the parity tests (one float32 rounding)."""
import numpy as np
import pytest

import datagen
from oracle import draft as OD

from gpu_util import say, to_host
from test_gpu_draft import Batch

pytestmark = pytest.mark.gpu


def reread(b):
    """The oracle's rows from the statistics on the device, after a test has changed them."""
    import invariant_token_log_fp32_amd as rlk

    def rows(old, t, stats):
        part, thr, status = (to_host(f.contiguous()) for f in rlk.support_state_fields(stats[3]))
        return old._replace(temperature=t, policy=to_host(stats[0]), lse_support=part, threshold=thr, status=status)

    b.rows = rows(b.rows, b.t, b.stats)
    if b.qlg is not None:
        b.q_rows = rows(b.q_rows, b.tq, b.qstats)


def likely(b):
    """Drafted tokens that are the drafter's maxima."""
    b.token[:] = [int(np.argmax(OD.decode_bf16(q[:b.vr]))) for q in b.q_bits]


# sequences that share a workgroup's work out, one workgroup each, and half a compute unit each
@pytest.mark.parametrize("times", [1, 17, 33])
@pytest.mark.parametrize("accept_u", [0.0, 1 - 2.0 ** -53])
def test_a_row_without_a_policy_ends_its_sequence(times, accept_u):
    """NaN in either field of a record, an infinite lse_support, a temperature
    that is none: in the first row, in a row behind accepted tokens, in the row
    behind the last drafted token, on either side."""
    import torch
    say(f"case: rows without a policy, {8 * times} sequences, accept_u {accept_u}")
    b = Batch(np.random.default_rng(31), [2] * 8 * times, 2100, 2112, (1.0,), 0.9, -1, "sampled")
    b.bits[1::3] = b.bits[0::3]
    b.q_bits[0::2] = b.bits[0::3]        # equal rows: drafted tokens before the changed row stay
    b.q_bits[1::2] = b.bits[1::3]
    likely(b)
    for s in range(7, 8 * times, 8):     # greedy targets, whose records hold NaN, are served
        b.t[3 * s:3 * s + 3] = 0.0
    b.accept_u[:] = accept_u
    b.score()
    tr, qr = b.stats[3].view(torch.float32), b.qstats[3].view(torch.float32)
    for s in range(0, 8 * times, 8):
        tr[3 * s, 1] = float("nan")                    # sequence 0: the first row's threshold
        tr[3 * (s + 1) + 1, 0] = float("nan")          # 1: the second row's lse_support
        tr[3 * (s + 2) + 2, 1] = float("nan")          # 2: the last row's threshold
        qr[2 * (s + 3), 1] = float("nan")              # 3: the draft's first row's threshold
        qr[2 * (s + 4) + 1, 0] = float("inf")          # 4: its second row's lse_support
        b.t[3 * (s + 5)] = np.nan                      # 5: temperatures
        b.tq[2 * (s + 6) + 1] = np.inf
    reread(b)
    got = b.check()
    for s in range(0, 8 * times, 8):
        at = [0, 1, 2, 0, 1, 0, 1]
        assert got[1][s:s + 7].tolist() == at
        for i, k in enumerate(at):
            row = 3 * (s + i) + k
            assert got[0][row] == -1 and np.isnan(got[2][row]) and np.isnan(got[3][row])
        assert got[0][3 * (s + 7)] >= 0


@pytest.mark.parametrize("times", [1, 33])
def test_a_greedy_draft_row_without_a_policy_ends_its_sequence(times):
    """Greedy rows of a drafter are point masses whose records hold NaN; one
    that the forward call refused (a status below 0, a NaN logprob) is none."""
    say(f"case: greedy draft rows without a policy, {4 * times} sequences")
    b = Batch(np.random.default_rng(32), [2] * 4 * times, 2100, 2112, (1.0,), 1.0, -1, "sampled")
    likely(b)
    b.tq[:] = 0.0
    b.accept_u[:] = 0.0
    b.q_bits[0::8, 9] = 0x7FC0                          # sequence 0: NaN in the draft's first row
    b.score()
    b.qstats[3][3::8, 2] = -1                           # 1: a status of the second row
    b.qstats[0][4::8] = float("nan")                    # 2: a logprob of the first row; 3 is served
    reread(b)
    assert b.q_rows.status[0] == -2 and np.isnan(b.q_rows.policy[0])
    got = b.check()
    for s in range(0, 4 * times, 4):
        assert got[1][s:s + 4].tolist() == [0, 1, 0, 2]
        for i, k in enumerate([0, 1, 0]):
            row = 3 * (s + i) + k
            assert got[0][row] == -1 and np.isnan(got[2][row]) and np.isnan(got[3][row])
        assert (got[0][3 * (s + 3):3 * (s + 3) + 3] >= 0).all()


@pytest.mark.parametrize("n,kind", [(5, "none"), (140, "none"), (5, "point"), (140, "point"), (5, "sampled"), (140, "sampled")])
@pytest.mark.parametrize("above", [500.0, 800.0, 2e9, 3e9, 1e12])
def test_weights_beyond_float64(n, kind, above):
    """A record whose lse_support lies far below a column's logit: e^500 can be
    drawn from, e^800 and more is no weight and refuses the sequence, whatever
    an integer of its exponent would wrap to; also where the drafter's weight
    of that column is as large."""
    import torch
    say(f"case: weights of e^{above:g}, {n} sequences, drafter {kind}")
    vr, vp = 40000, 40064
    b = Batch(np.random.default_rng(33), [0 if kind == "none" else 1] * n, vr, vp, (1.0,), 1.0, -1,
              "sampled" if kind == "sampled" else "point")
    big = datagen.f32_to_bf16_bits(np.array([above], np.float32))[0]
    step = 1 if kind == "none" else 2
    b.bits[::step, 777] = big
    b.accept_u[:] = 1 - 2.0 ** -53
    b.token[:] = 5
    b.q_bits[:, 777] = big
    b.score()
    b.stats[3].view(torch.float32)[:, 0] = 0.0          # as if the large column were none
    b.stats[0][:] = -60.0
    if kind == "sampled":
        b.qstats[3].view(torch.float32)[:, 0] = 0.0
        b.qstats[0][:] = -1.0
    reread(b)
    got = b.check()
    if kind == "sampled" and above == 500.0:            # equal weights of that column: drawn among the others
        assert (got[0][::step] >= 0).all() and (got[0][::step] != 777).all()
    else:
        assert (got[0][::step] == (777 if above == 500.0 else -1)).all()


@pytest.mark.parametrize("counts", [[0] * 40, [2] * 40, [1] * 200])
def test_tiny_temperatures(counts):
    """Temperatures down to a subnormal one: the oracle's tokens, or its refusal
    where the forward call's float32 statistics give no finite weight."""
    say(f"case: tiny temperatures, {len(counts)} sequences of {max(counts)} drafted tokens")
    b = Batch(np.random.default_rng(34), counts, 3000, 3008, (1e-4, 1e-8, 1e-10, 1e-12, 1e-17, 1e-40), 1.0, -1, "sampled")
    likely(b)
    got = b.score().check()
    sharp = (b.t == np.float32(1e-4)) & (got[0] >= 0)
    assert sharp.any()


@pytest.mark.parametrize("n", [4, 140])
def test_weights_that_sum_to_0(n):
    """An lse_support far above every logit: no weight is left, and a refused
    drafted token comes out if it has a logprob."""
    import torch
    say(f"case: weights that sum to 0, {n} sequences")
    b = Batch(np.random.default_rng(35), [1, 1, 1, 0] * (n // 4), 9000, 9024, (1.0,), 1.0, -1, "point").score()
    b.accept_u[:] = 0.5
    b.stats[3].view(torch.float32)[:, 0] = 1000.0
    b.stats[0][:] = -900.0
    b.stats[0][2::7] = float("-inf")     # the second sequence of four: rows 2 and 3 of seven
    reread(b)
    got = b.check()
    for s in range(0, n, 4):
        row = 7 * (s // 4)
        assert got[0][row] == b.token[3 * (s // 4)] and got[0][row + 4] == b.token[3 * (s // 4) + 2]
        assert (got[0][[row + 2, row + 6]] == -1).all() and np.isnan(got[2][[row + 2, row + 6]]).all()
