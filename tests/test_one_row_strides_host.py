"""Matrices of one row (or none): the row stride has no meaning, so any is taken. Such views
are the last position of a sequence, hidden[:, -1] of a [1, length, d] tensor, whose stride
is length * d. Host tests of what the binding passes on (no kernel is launched)."""
import pytest
import torch

import invariant_token_log_fp32_amd as rlk

META = torch.device("meta")
LIMIT = 1 << 21  # the largest row stride that the entry points take


def view(n, d, stride, dtype=torch.bfloat16):
    return torch.empty((n + 1) * stride + d, dtype=dtype, device=META).as_strided((n, d), (stride, 1))


class OnGpu(torch.Tensor):
    """A meta tensor that passes for a device tensor."""

    is_cuda = True


def device_view(*args):
    return view(*args).as_subclass(OnGpu)


@pytest.mark.parametrize("n", [0, 1])
@pytest.mark.parametrize("stride", [64, 67, 4 * LIMIT, 4 * LIMIT + 3])
def test_any_stride_of_one_row(n, stride):
    for t, kind in ((torch.bfloat16, rlk.TYPE_BF16), (torch.float32, rlk.TYPE_F32)):
        assert rlk._matrix(view(n, 64, stride, t), "x") == (64, kind)
        v = view(n, 64, stride, t)
        assert rlk._grad_out(v, (n, 64), torch.bfloat16, META, "grad_hidden") is v
    assert rlk._bf16_matrix(device_view(n, 64, stride), "hidden") == 64


def test_the_stride_of_one_row_of_logits_is_kept():
    """vocab_padded columns are read, which may be more than the view has: its stride says
    that they are there."""
    assert rlk._check_logits(device_view(1, 1000, 1024)) == 1024
    assert rlk._check_logits(device_view(1, 1024, 1000)) == 1024


@pytest.mark.parametrize("stride", [64, 72, 4 * LIMIT, 67])
def test_the_stride_of_several_rows_is_passed_on(stride):
    assert rlk._matrix(view(2, 64, stride), "x")[0] == stride
    assert rlk._bf16_matrix(device_view(2, 64, stride), "hidden") == stride
    assert rlk._check_logits(device_view(2, 64, stride)) == stride
    v = view(2, 64, stride)
    if stride % 8:
        with pytest.raises(ValueError, match="multiple of 8"):
            rlk._grad_out(v, (2, 64), torch.bfloat16, META, "grad_hidden")
    else:
        assert rlk._grad_out(v, (2, 64), torch.bfloat16, META, "grad_hidden") is v
