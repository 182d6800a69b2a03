"""The oracle of the verification on records that cannot be served: a row
reached whose record, policy logprob or temperature is no number ends its
sequence with token -1, whichever side it is on and whether or not its drafted
token would have stayed."""
import numpy as np
import pytest

from oracle import draft as OD
from test_draft_host import scored


def one(side, field, value, place, accept_u):
    """A sequence of two drafted tokens, equal rows on both sides; one field of row `place` of a side is changed."""
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (3, 12))
    t, d = scored(x, 0.8, [2, 5, 0]), scored(x[:2], 0.8, [2, 5])
    rows = t if side == "target" else d
    changed = getattr(rows, field).copy()
    changed[place] = value
    rows = rows._replace(**{field: changed})
    t, d = (rows, d) if side == "target" else (t, rows)
    return OD.verify(t, d, 12, [0, 2], [2, 5], [accept_u, accept_u], [0.5])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("accept_u", [0.0, 1 - 2.0 ** -53])
@pytest.mark.parametrize("field,value", [("threshold", NAN), ("lse_support", NAN), ("lse_support", INF), ("lse_support", -INF),
                                         ("temperature", NAN), ("temperature", INF), ("temperature", -1.0), ("status", -1),
                                         ("status", -2)])
@pytest.mark.parametrize("side,place", [("target", 0), ("target", 1), ("target", 2), ("draft", 0), ("draft", 1)])
def test_a_row_without_a_policy_ends_its_sequence(side, place, field, value, accept_u):
    out, accepted, policy, ref, margin = one(side, field, value, place, accept_u)
    assert accepted[0] == place                 # equal rows: every drafted token before it stays
    assert out[place] == -1 and np.isnan(policy[place]) and np.isnan(ref[place])
    assert (out[place + 1:] == -1).all() and (policy[place + 1:] == 0).all() and margin[0] == INF


@pytest.mark.parametrize("field,value,served", [("status", -1, False), ("status", -2, False), ("policy", NAN, False),
                                                ("lse_support", NAN, True), ("policy", -INF, True)])
@pytest.mark.parametrize("place", [0, 1])
def test_a_greedy_draft_row_is_a_point_mass_if_it_has_a_policy(place, field, value, served):
    x = np.random.default_rng(2).normal(0, 1, (3, 12))
    t, d = scored(x, 0.8, [2, 5, 0]), scored(x[:2], 0.8, [2, 5])
    d = d._replace(temperature=np.zeros(2, np.float32), policy=np.zeros(2, np.float32), lse_support=np.full(2, NAN, np.float32))
    changed = getattr(d, field).copy()
    changed[place] = value
    out, accepted, policy, _, _ = OD.verify(t, d._replace(**{field: changed}), 12, [0, 2], [2, 5], [0.0, 0.0], [0.5])
    assert accepted[0] == (2 if served else place)
    assert served or (out[place] == -1 and np.isnan(policy[place]))
    assert not served or out[2] >= 0


@pytest.mark.parametrize("kind", ["none", "point", "drafter"])
@pytest.mark.parametrize("part,drawn", [(0.0, True), (-500.0, True), (-800.0, False), (-2e9, False), (800.0, False), (2e9, False)])
def test_sums_that_are_not_finite_are_not_drawn_from(kind, part, drawn):
    """lse_support far below the logits: weights up to e^500 are drawn from, an
    infinite sum is not, nor is a row whose weights all vanish."""
    x = np.random.default_rng(3).normal(0, 1, (2, 12))
    t = scored(x, 1.0, [2, 0])
    t = t._replace(lse_support=np.full(2, part, np.float32), policy=np.full(2, -np.inf if part > 0 else -60.0, np.float32))
    d = scored(x[:1], 1.0, [2])
    d = d._replace(lse_support=np.full(1, part + 1 if drawn else part, np.float32), policy=np.zeros(1, np.float32))
    count = 0 if kind == "none" else 1
    out, accepted, policy, _, margin = OD.verify(t, d if kind == "drafter" else None, 12, [0, count], [2] * count,
                                                 [1 - 2.0 ** -53] * count, [0.5])
    assert accepted[0] == 0
    if drawn:
        assert out[0] >= 0 and margin[0] < 1
    else:
        assert out[0] == -1 and np.isnan(policy[0]) and margin[0] == INF


@pytest.mark.parametrize("logp,token", [(-900.0, 2), (-INF, -1)])
def test_weights_that_sum_to_0_leave_the_drafted_token_if_it_has_a_logprob(logp, token):
    x = np.random.default_rng(4).normal(0, 1, (2, 12))
    t = scored(x, 1.0, [2, 0])
    t = t._replace(lse_support=np.full(2, 1000.0, np.float32), policy=np.full(2, logp, np.float32))
    out, accepted, policy, _, _ = OD.verify(t, None, 12, [0, 1], [2], [0.5], [0.5])
    assert accepted[0] == 0 and out[0] == token and (policy[0] == logp if token >= 0 else np.isnan(policy[0]))
