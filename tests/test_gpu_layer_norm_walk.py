"""The norms' walks over many rows: workgroups of 2, 4 and 8 waves that go through at least
four rows each, forward and backward, live rows and padding in turn, against the float64
oracle.

Rows a workgroup: forward ceil(n / w) with w = 256 compute units times the workgroups of
2048 threads, backward with 768 or, above 2^25 values, 512 threads; `walks` says how many and
the test asserts at least four.

Tolerances of the forward pass and of dx: those of test_gpu_layer_norm.py (their sums are
the same, whatever the rows of a workgroup). dweight and dbias, u = 2^-24: each term is off
by 3 u; a column is added over a workgroup's rows (at most ceil(n / 256) additions), then by
a thread over its share of at most 3072 workgroups (in four sums, at most 3 additions of
eights and 7 of the rest), 2 and 5 additions to join those: n / 256 + 80 covers them all,
counted in u of the sum of the magnitudes.
"""
import numpy as np
import pytest

import invariant_token_log_fp32_amd as rlk
from oracle import layer_norm as LN

from gpu_util import say, to_host
from test_gpu_layer_norm import U, check, check_forward, make, vector

pytestmark = pytest.mark.gpu


def walks(n, d):
    """(waves, rows of a workgroup forward, backward)"""
    a_wave = (2 if d <= 8192 else 4) * 512  # values
    waves = -(-d // a_wave)

    def rows(threads):
        return -(-n // (256 * max(1, threads // (64 * waves))))

    return waves, rows(2048), rows(512 if n * d > 1 << 25 else 768)


# n, d, waves, more than 2^25 values
SIZES = [(13000, 1032, 2, False), (33000, 1032, 2, True), (7000, 3080, 4, False), (11000, 3080, 4, True), (3500, 7304, 8, False),
         (3100, 14400, 8, True)]
KINDS = [(False, True, True), (True, False, False), (False, True, False)]  # rms, x32, w32


@pytest.mark.parametrize("n,d,waves,large", SIZES)
@pytest.mark.parametrize("rms,x32,w32", KINDS[:2])
def test_forward(n, d, waves, large, rms, x32, w32):
    import torch
    say(f"case: forward walk {n} x {d}, rms {rms}, x32 {x32}, w32 {w32}")
    assert walks(n, d)[0] == waves and walks(n, d)[1] >= 4
    rng = np.random.default_rng(n)
    x, xv = make(rng, n, d, x32, pad=8, scale=np.exp2(rng.integers(-6, 7, (n, 1))), offset=0.5)
    w, wv = vector(rng, d, w32)
    b, bv = vector(rng, d, w32, 0.0)
    y, mean, rstd = rlk.layer_norm(x, w, b, rms=rms, eps=1e-5, return_stats=True)
    check_forward(y, mean, rstd, xv, wv, bv, 1e-5, rms)
    if not x32:
        out = rlk.layer_norm(x, w, b, rms=rms, eps=1e-5, out=x)  # in place: the next row is loaded before this one is stored
        assert out is x and torch.equal(x, y)


@pytest.mark.parametrize("n,d,waves,large", SIZES)
@pytest.mark.parametrize("rms,x32,w32", KINDS)
def test_backward(n, d, waves, large, rms, x32, w32):
    """Half of the rows are padding that holds NaN, so live and empty rows meet at every
    distance in a workgroup; an eighth of the live rows have one value of dy alone."""
    import torch
    say(f"case: backward walk {n} x {d}, rms {rms}, x32 {x32}, w32 {w32}")
    assert walks(n, d)[0] == waves and walks(n, d)[2] >= 4 and (n * d > 1 << 25) == large
    rng = np.random.default_rng(n + 1)
    x, xv = make(rng, n, d, x32, pad=8, scale=np.exp2(rng.integers(-3, 4, (n, 1))), offset=0.5)
    w, wv = vector(rng, d, w32)
    dy, dyv = make(rng, n, d, False)
    empty = rng.random(n) < 0.5
    lone = ~empty & (rng.random(n) < 0.125)
    keep = np.zeros((int(lone.sum()), d), bool)
    keep[np.arange(len(keep)), rng.integers(0, d, len(keep))] = True
    dyv[empty] = 0
    dyv[lone] = np.where(keep, dyv[lone], 0)
    dy.copy_(torch.from_numpy(dyv))  # (BF16 values: exact)
    _, m, r = LN.forward(xv, wv, None, 1e-5, rms)
    m, r = m.astype(np.float32).astype(np.float64), r.astype(np.float32).astype(np.float64)
    mean, rstd = (torch.from_numpy(v.astype(np.float32)).to("cuda:0") for v in (m, r))
    off = torch.from_numpy(empty).to("cuda:0")
    for v in (x, mean, rstd):
        v[off] = float("nan")
    dx, dw, db = rlk.layer_norm_backward(dy, x, w, None if rms else mean, rstd, rms=rms, bias_grad=True)
    want_dx, want_dw, want_db = LN.backward(dyv, xv, wv, m, r, rms)
    hat = (xv - (0 if rms else m[:, None])) * r[:, None]
    g = np.abs(dyv * wv)
    c1 = 0 if rms else g.mean(1, keepdims=True)
    c2 = (g * np.abs(hat)).mean(1, keepdims=True)
    hat = np.abs(hat)
    tol = r[:, None] * U * (8 * g + 44 * c1 + 48 * hat * c2) + (2 * U if x32 else 2.0 ** -8) * np.abs(want_dx) + 1e-40
    check(dx, want_dx, tol, "dx")
    assert bool((dx[off] == 0).all())
    check(dw, want_dw, (n / 256 + 80) * U * (np.abs(dyv) * hat).sum(0) + 1e-45, "dweight")
    check(db, want_db, (n / 256 + 80) * U * np.abs(dyv).sum(0) + 1e-45, "dbias")
    # in place and without the bias' sums: the same bytes
    dx2, dw2, _ = rlk.layer_norm_backward(dy, x, w, None if rms else mean, rstd, rms=rms, grad_x=x)
    assert dx2 is x and torch.equal(dx2, dx) and torch.equal(dw2, dw)
