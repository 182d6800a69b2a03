"""The serving bindings keep layouts and sizes between calls by value, never by
an object's identity. CPU only: the tensors are host tensors and the entry
points' calls are recorded instead of made."""
import numpy as np
import pytest
import torch

import invariant_token_log_fp32_amd as rlk


@pytest.fixture
def calls(monkeypatch):
    """(name, layout, bytes of workspace) of each call that would be made."""
    made = []

    def run(name, device, *args):
        layout = next(a._obj for a in args if isinstance(getattr(a, "_obj", None), rlk.VocabLayout))
        made.append((name, layout.vocab_padded, layout.vocab_real, args[-1]))

    monkeypatch.setattr(rlk, "_run", run)
    monkeypatch.setattr(rlk, "_check_logits", lambda x: x.stride(0))
    monkeypatch.setattr(rlk, "_bf16_matrix", lambda x, name: x.stride(0))
    return made


@pytest.mark.parametrize("make", [torch.tensor, np.array])
def test_sizes_given_as_arrays_whose_values_change(calls, make):
    real, padded = make(1000), make(2048)
    hidden = torch.zeros((3, 64), dtype=torch.bfloat16)
    codes, scales = (torch.zeros(n, dtype=torch.uint8) for n in rlk.mx4_bytes(2048, 64))
    logits = torch.zeros((3, 2048), dtype=torch.bfloat16)
    f, start = torch.zeros(3), torch.arange(4) * 0
    none = torch.zeros(0, dtype=torch.int64)

    def both():
        rlk.mx4_linear(hidden, codes, scales, vocab_real=real, vocab_padded=padded)
        rlk.draft_verify(logits, none, start, none.double(), f.double(), temperature=1.0, policy_logp=f, ref_logp=f, lse=f,
                         support_state=torch.zeros((3, 4), dtype=torch.int32), vocab_real=real, vocab_padded=padded)

    both()
    real[()] = 2000
    both()
    linear = sum(rlk.mx4_bytes(3, 64))
    assert calls == [("rlk_mx4_linear", 2048, 1000, linear), ("rlk_draft_verify", 2048, 1000, 3 * 2 * 8),
                     ("rlk_mx4_linear", 2048, 2000, linear), ("rlk_draft_verify", 2048, 2000, 3 * 4 * 8)]
