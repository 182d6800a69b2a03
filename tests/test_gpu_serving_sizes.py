"""The serving operators at the largest and the odd sizes that their headers
allow. The products' inputs are grid values whose sums float32 holds exactly
in any order (asserted by the sum of the magnitudes), so every logit is
compared with the exact sum rounded once to BF16."""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import mx4 as MX

from gpu_util import say, to_host
from test_gpu_draft import Batch, dev
from test_gpu_mx4 import exact_matrix, run_linear

pytestmark = pytest.mark.gpu


def exact_logits(hb, wb):
    h, w = MX.decode_bf16(hb).astype(np.float32), MX.decode_bf16(wb).astype(np.float32)
    assert (np.abs(h) @ np.abs(w).T).max() * 4 < 2 ** 24   # quarters
    return datagen.f32_to_bf16_bits(h @ w.T)


@pytest.mark.parametrize("n", [1, 33, 130, 300])
def test_linear_at_the_longest_d(n):
    say(f"case: exact 4-bit linear {n} x 65536 x 300")
    rng = np.random.default_rng(n)
    hb, wb = exact_matrix(rng, n, 65536, 0.5), exact_matrix(rng, 300, 65536, 0.5)
    assert np.array_equal(run_linear(hb, wb, 320), exact_logits(hb, wb))


@pytest.mark.parametrize("n", [2, 40])
def test_linear_at_the_widest_stride_of_hidden_states(n):
    say(f"case: exact 4-bit linear {n} x 96 x 500, stride 2^21")
    rng = np.random.default_rng(n)
    hb, wb = exact_matrix(rng, n, 96), exact_matrix(rng, 500, 96)
    assert np.array_equal(run_linear(hb, wb, 512, hpad=2 ** 21 - 96), exact_logits(hb, wb))


@pytest.mark.parametrize("n", [3, 40, 100, 300, 1030])
@pytest.mark.parametrize("d", [64, 800, 4640])
def test_linear_of_pad_columns_behind_a_few_real_ones(n, d):
    """Whole tiles of pad columns: -inf there (checked by run_linear), the projection's last tile read again."""
    say(f"case: exact 4-bit linear {n} x {d} x 37/20032")
    rng = np.random.default_rng(n + d)
    hb, wb = exact_matrix(rng, n, d), exact_matrix(rng, 37, d)
    assert np.array_equal(run_linear(hb, wb, 20032), exact_logits(hb, wb))


def device_exact(gen, n, d):
    """Grid values on the device, 6 in every block: their own 4-bit values at scale 1."""
    import torch
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.bfloat16, device="cuda:0")
    v = grid[torch.randint(0, 8, (n, d), generator=gen, device="cuda:0")]
    v *= (torch.randint(0, 2, (n, d), generator=gen, device="cuda:0") * 2 - 1).to(torch.bfloat16)
    v[:, ::32] = 6.0
    return v


@pytest.mark.parametrize("n,vr,vp", [(2, 1 << 22, 1 << 22), (40, (1 << 22) - 5, 1 << 22), (130, (1 << 22) - 33, 1 << 22),
                                     (1 << 22, 61, 64)])
def test_the_largest_matrices(n, vr, vp):
    """2^22 rows of the projection, 2^22 hidden states: the codes of a part alone are those of the whole, and every logit is exact."""
    import torch
    say(f"case: exact 4-bit linear {n} x 32 x {vr}")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(n)
    h, w = device_exact(gen, n, 32), device_exact(gen, vr, 32)
    wc, ws = rlk.mx4_quantize(w)
    large = h if n > vr else w
    codes, scales, v = rlk.mx4_quantize(large, return_values=True)
    assert torch.equal(v, large)
    at = (large.shape[0] // 2) // 32 * 32
    c2, s2 = rlk.mx4_quantize(large[at:].contiguous())
    first = rlk.mx4_bytes(at, 32)
    assert torch.equal(codes[first[0]:], c2) and torch.equal(scales[first[1]:], s2)
    out = rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp)
    for r in range(0, n, 1 << 20):   # products below 2^31 bytes: torch's of more came back with zeros at the end
        for c in range(0, vr, 1 << 20):
            want = (h[r:r + (1 << 20)].float() @ w[c:c + (1 << 20)].float().t()).to(torch.bfloat16)
            assert torch.equal(out[r:r + (1 << 20), c:min(vr, c + (1 << 20))], want)
    assert (out[:, vr:] == float("-inf")).all()


@pytest.mark.parametrize("n", [6, 200])
def test_draft_rows_of_another_stride_and_more_than_drafted(n):
    """The drafter's rows in a wider buffer than the target's, with rows behind the last drafted token that hold NaN."""
    import torch
    say(f"case: {n} sequences, draft rows of another stride, five to spare")
    b = Batch(np.random.default_rng(n), [2] * n, 3001, 3008, (0.8, 0.0), 0.95, -1, "sampled").score()
    want = [w.tobytes() for w in b.check()]
    nd = len(b.token)
    wide = torch.full((nd + 5, 3008 + 72), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide[:nd, :3008] = b.qlg

    def longer(t):
        out = torch.full((nd + 5,) + tuple(t.shape[1:]), -1, dtype=t.dtype, device="cuda:0")
        out[:nd] = t
        return out

    pol, ref, lse, state = b.stats
    got = rlk.draft_verify(b.lg, dev(b.token), dev(b.start), dev(b.accept_u), dev(b.sample_u), temperature=dev(b.t),
                           policy_logp=pol, ref_logp=ref, lse=lse, support_state=state, vocab_real=3001, vocab_padded=3008,
                           draft_logits=wide, draft_temperature=longer(dev(b.tq)), draft_policy_logp=longer(b.qstats[0]),
                           draft_support_state=longer(b.qstats[3]))
    torch.cuda.synchronize()
    assert [to_host(g).tobytes() for g in got] == want


@pytest.mark.parametrize("counts,temps", [([1], (1.0,)), ([0, 2], (0.5, 0.0))])
def test_a_vocabulary_of_millions(counts, temps):
    say(f"case: {len(counts)} sequences of 3000001 columns")
    Batch(np.random.default_rng(41), counts, 3000001, 3000064, temps, 0.999, -1, "sampled").score().check()
