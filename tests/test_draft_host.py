"""Host tests of the verification of drafted tokens: the oracle keeps the
target's distribution (exactly, by enumeration), the C ABI's refusals (fake
device addresses, nothing is launched) and the binding's checks."""
import ctypes

import numpy as np
import pytest
import torch

import datagen
import invariant_token_log_fp32_amd as rlk
from invariant_token_log_fp32_amd import ScoredRows, VocabLayout
from oracle import draft as OD

OK, NULL, ALIGN, SHAPE, GROUPS, WS = 0, -1, -2, -3, -4, -5
P = 0x100000


def scored(x, t, token, threshold=None):
    """Rows of the oracle with float64 statistics rounded to float32."""
    bits = datagen.f32_to_bf16_bits(np.asarray(x, np.float32))
    n = len(bits)
    v = OD.decode_bf16(bits)
    thr = np.full(n, -np.inf, np.float32) if threshold is None else np.asarray(threshold, np.float32)
    z = (v.astype(np.float32) / np.float32(t)).astype(np.float64)
    inside = v >= thr[:, None]
    part = np.log(np.where(inside, np.exp(z), 0).sum(1))
    full = np.log(np.exp(z).sum(1))
    zt, hit = z[np.arange(n), token], inside[np.arange(n), token]
    return OD.Rows(bits, np.full(n, t, np.float32), np.where(hit, zt - part, -np.inf).astype(np.float32),
                   part.astype(np.float32), thr, hit.astype(np.int32), (zt - full).astype(np.float32),
                   full.astype(np.float32))


@pytest.mark.parametrize("kind", ["drafter", "point"])
def test_oracle_emits_the_targets_distribution(kind):
    """One drafted token over a vocabulary of 9, the random numbers on a grid:
    the emitted first tokens' frequencies, weighted by the drafter's
    probabilities, are the target's policy to within the grid's step."""
    rng = np.random.default_rng(2)
    v, grid = 9, 64
    px, qx = rng.normal(0, 1.5, (1, v)), rng.normal(0, 1.5, (1, v))
    seen = np.zeros(v)
    want = OD.distribution(scored(px, 0.8, [0]), 0, v)
    q = OD.distribution(scored(qx, 1.1, [0]), 0, v) if kind == "drafter" else None
    for d in ([*range(v)] if kind == "drafter" else [3]):
        t = scored(np.concatenate((px, px)), 0.8, [d, 0])
        dr = scored(qx, 1.1, [d]) if kind == "drafter" else None
        for a in range(grid):
            for b in range(grid):
                out = OD.verify(t, dr, v, [0, 1], [d], [(a + 0.5) / grid], [(b + 0.5) / grid])
                assert out[1][0] in (0, 1) and (out[1][0] == 0 or out[0][0] == d)
                seen[out[0][0]] += (q[d] if q is not None else 1.0) / grid ** 2
    # each accept border lies within half a step, each drawing border within one
    assert np.abs(seen - want).max() <= 2.0 / grid
    assert abs(seen.sum() - 1) < 1e-6


def test_oracle_special_cases():
    x = np.array([[0.0, 1.0, 2.0, 2.0], [0.0, 1.0, 2.0, 2.0]])
    t = scored(x, 1.0, [1, 0])
    # equal rows: accepted whatever the number below 1
    same = scored(x[:1], 1.0, [1])
    assert OD.verify(t, same, 4, [0, 1], [1], [1 - 2.0 ** -53], [0.5])[1][0] == 1
    # p nowhere above q and yet refused (a rounded statistic): the drafted token itself
    off = same._replace(policy=np.array([0.0], np.float32))
    out = OD.verify(t, off, 4, [0, 1], [1], [0.9], [0.5])
    assert out[1][0] == 0 and out[0].tolist() == [1, -1] and out[2][0] == t.policy[0]
    # greedy: the lowest column of the maximum
    g = t._replace(temperature=np.zeros(2, np.float32), policy=np.array([-np.inf, 0], np.float32))
    out = OD.verify(g, None, 4, [0, 1], [1], [0.0], [0.99])
    assert out[0].tolist() == [2, -1] and out[2][0] == 0.0
    # offsets out of order, out of range
    assert OD.verify(t, None, 4, [1, 0], [1], [0.0], [0.5])[1][0] == -1
    assert OD.verify(t, None, 4, [0, 2], [1], [0.0], [0.5])[1][0] == -1


class Call:
    """One call with fake addresses; keyword arguments change one thing each."""

    def __init__(self, **kw):
        self.t = dict(logits=P, n_rows=9, row_stride=1024, temperature=2 * P, policy_logp=3 * P, ref_logp=4 * P,
                      lse=5 * P, support=6 * P)
        self.d = dict(logits=7 * P, n_rows=6, row_stride=1024, temperature=8 * P, policy_logp=9 * P, ref_logp=None,
                      lse=None, support=10 * P)
        self.a = dict(n_seq=3, n_draft=6, start=11 * P, token=12 * P, accept=13 * P, sample=14 * P, tok=15 * P,
                      acc=16 * P, pol=17 * P, ref=18 * P, ws=19 * P, wsb=1 << 16)
        self.layout = VocabLayout(1024, 1000, 1024, 8, 1)
        for k, v in kw.items():
            if k[:2] in ("t_", "d_"):
                (self.t if k[0] == "t" else self.d)[k[2:]] = v
            elif k == "layout":
                self.layout = v
            elif k in ("target", "draft"):
                setattr(self, k[0], v)
            else:
                self.a[k] = v

    def __call__(self):
        a = self.a
        rows = [None if r is None else ctypes.byref(ScoredRows(**r)) for r in (self.t, self.d)]
        return rlk.load_library().rlk_draft_verify(
            rows[0], rows[1], ctypes.byref(self.layout) if self.layout is not None else None, a["n_seq"], a["n_draft"],
            a["start"], a["token"], a["accept"], a["sample"], a["tok"], a["acc"], a["pol"], a["ref"], a["ws"], a["wsb"],
            None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, NULL) for k in ("target", "layout", "t_logits", "t_temperature", "t_policy_logp", "t_ref_logp", "t_lse",
                                  "t_support", "d_logits", "d_temperature", "d_policy_logp", "d_support", "start",
                                  "token", "accept", "sample", "tok", "acc", "pol", "ref", "ws")],
    *[({k: P + 8}, ALIGN) for k in ("t_logits", "d_logits", "ws")],
    *[({k: P + 4}, ALIGN) for k in ("start", "token", "accept", "sample", "tok")],
    *[({k: P + 2}, ALIGN) for k in ("t_temperature", "t_policy_logp", "t_ref_logp", "t_lse", "t_support", "d_temperature",
                                    "d_policy_logp", "d_support", "acc", "pol", "ref")],
    (dict(t_n_rows=8), SHAPE), (dict(d_n_rows=5), SHAPE), (dict(t_row_stride=1016), SHAPE), (dict(d_row_stride=1028), SHAPE),
    (dict(t_n_rows=(1 << 23) + 1), SHAPE), (dict(t_row_stride=1 << 61), SHAPE),
    (dict(n_seq=-1), SHAPE), (dict(n_draft=-1), SHAPE), (dict(n_seq=(1 << 22) + 1, t_n_rows=1 << 23), SHAPE),
    (dict(layout=VocabLayout(1000, 1000, 1024, 8, 1)), SHAPE), (dict(layout=VocabLayout(1024, 0, 1024, 8, 1)), SHAPE),
    (dict(layout=VocabLayout(1024, 1000, 1024, 8, 5)), GROUPS), (dict(wsb=3 * 2 * 8 - 1), WS),
])
def test_verify_refuses(kw, code):
    assert Call(**kw)() == code


def test_no_sequences_enqueue_nothing():
    assert Call(n_seq=0, n_draft=0, t_logits=None, start=None, tok=None, ws=None, draft=None, wsb=0)() == OK
    assert Call(n_seq=0, layout=VocabLayout(1024, 1000, 1024, 8, 3))() == GROUPS


def test_workspace_size():
    assert rlk.draft_workspace_bytes(3, 1024, 1000) == 3 * 2 * 8
    assert rlk.draft_workspace_bytes(7, 152576, 151936) == 7 * 297 * 8
    assert rlk.draft_workspace_bytes(7, 4096, 512) == 7 * 8 and rlk.draft_workspace_bytes(7, 4096, 513) == 7 * 16
    assert rlk.draft_workspace_bytes(-1, 1024, 1000) == 0 and rlk.draft_workspace_bytes(3, 1000, 1000) == 0


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(ScoredRows) == 64
    assert [f[0] for f in ScoredRows._fields_] == ["logits", "n_rows", "row_stride", "temperature", "policy_logp",
                                                   "ref_logp", "lse", "support"]


def test_binding_checks_inputs():
    meta = torch.device("meta")
    ok = torch.empty(4, dtype=torch.int64, device=meta)
    rlk._given(meta, (ok, (4,), torch.int64, "draft_token"), (ok, (4,), torch.int64, "again"))
    for bad in (None, 3, ok.int(), ok[:3], torch.empty(8, dtype=torch.int64, device=meta)[::2],
                torch.empty(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            rlk._given(meta, (ok, (4,), torch.int64, "first"), (bad, (4,), torch.int64, "draft_token"))
