"""Host tests of the microscaled 4-bit operators: the oracle's pins, the C
ABI's refusals (fake device addresses; every call returns before a HIP call)
and the binding's argument checks. No GPU needed, no kernel is launched."""
import ctypes

import numpy as np
import pytest
import torch

import datagen
import invariant_token_log_fp32_amd as rlk
from invariant_token_log_fp32_amd import VocabLayout
from oracle import mx4 as MX

OK, NULL, ALIGN, SHAPE, GROUPS, WS = 0, -1, -2, -3, -4, -5
P = 0x10000
META = torch.device("meta")


def bits_of(values):
    return datagen.f32_to_bf16_bits(np.asarray(values, dtype=np.float32))


def test_oracle_rounds_to_the_nearest_grid_value_ties_to_even():
    """A block whose scale is 2^0 (its maximum is 4): every multiple of 1/64 up
    to 8 against the nearest of the eight magnitudes, found by enumeration."""
    x = np.arange(0, 7.9, 1 / 64)
    for sign in (1.0, -1.0):
        for v in x:
            row = np.zeros((1, 32), np.float32)
            row[0, 0], row[0, 7] = 4.0, sign * v
            bits = bits_of(row)
            v8 = abs(float(MX.decode_bf16(bits)[0, 7]))
            code, byte = MX.quantize(bits)
            assert byte[0, 0] == 127  # also when v > 4: floor(log2 v) is 2 up to 8
            off = [abs(v8 - g) for g in MX.GRID]
            best = [k for k in range(8) if off[k] == min(off)]
            want = best[0] if len(best) == 1 else [k for k in best if k % 2 == 0][0]
            assert code[0, 7] & 7 == want, v8
            assert (code[0, 7] >> 3) == (1 if sign < 0 else 0)


def test_oracle_scales_and_special_blocks():
    rows = np.zeros((9, 32), np.float32)
    rows[1, 3] = 1.0
    rows[2, 3] = 6.0
    rows[3, 3] = 2.0 ** -126
    rows[4, 3] = 2.0 ** -133          # a subnormal BF16
    rows[5, 3] = 3.0e38
    rows[6, 3] = np.nan
    rows[7, 3] = -np.inf
    rows[8, :] = -0.0
    code, byte = MX.quantize(bits_of(rows))
    assert byte[:, 0].tolist() == [0, 125, 127, 0, 0, 252, 255, 255, 0]
    v = MX.values(code, byte)
    assert v[1, 3] == 1.0 and v[2, 3] == 6.0 and v[3, 3] == 2.0 ** -126
    assert v[4, 3] == 0.0 and np.isnan(v[6]).all() and np.isnan(v[7]).all()
    assert v[5, 3] == 6.0 * 2.0 ** 125   # 2^127 * 1.76 is saturated
    assert (code[8] == 8).all()


def test_oracle_values_requantise_to_themselves():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (20, 96)) * np.exp2(rng.integers(-20, 20, (20, 1)))
    v = MX.values(*MX.quantize(bits_of(x)))
    again = MX.values(*MX.quantize(bits_of(v)))
    assert np.array_equal(v, again)
    # off by at most half a grid step below the saturation, 2 * 2^e above it
    e = MX.quantize(bits_of(x))[1].astype(np.int64) - 127
    assert np.all(np.abs(v - MX.decode_bf16(bits_of(x))).reshape(20, 3, 32) <= 2.0 ** (e[..., None] + 1))


def test_pack_places_every_block():
    rng = np.random.default_rng(4)
    n, d = 37, 288
    code, byte = rng.integers(0, 16, (n, d)).astype(np.uint8), rng.integers(1, 255, (n, d // 32)).astype(np.uint8)
    c, s = MX.pack(code, byte)
    assert (len(c), len(s)) == rlk.mx4_bytes(n, d)
    S = 4 * (-(-d // 256))
    for row, b in [(0, 0), (5, 1), (31, 8), (32, 3), (36, 8)]:
        st, h = b // 2, b % 2
        at = (((row // 32) * S + st) * 2 + h) * 512 + (row % 32) * 16
        got = c[at:at + 16]
        want = code[row, 32 * b:32 * b + 32]
        assert np.array_equal(got & 15, want[0::2]) and np.array_equal(got >> 4, want[1::2])
        assert s[(((row // 32) * S // 4 + st // 4) * 2 + h) * 128 + (row % 32) * 4 + st % 4] == byte[row, b]
    assert np.count_nonzero(s) == byte.size


def test_sizes():
    assert rlk.mx4_bytes(1, 32) == (4096, 256)
    assert rlk.mx4_bytes(33, 4096) == (2 * 16 * 4096, 2 * 16 * 256)
    assert rlk.mx4_bytes(0, 64) == (0, 0)
    for n, d in ((-1, 64), (1, 31), (1, 48), (1, 0), (1, 65568), ((1 << 22) + 1, 64)):
        assert rlk.mx4_bytes(n, d) == (0, 0)
        assert rlk.mx4_linear_workspace_bytes(n, d) == 0
    assert rlk.mx4_linear_workspace_bytes(40, 288) == sum(rlk.mx4_bytes(40, 288))


def test_every_declared_function_is_exported():
    lib = rlk.load_library()
    names = rlk.declared_functions(rlk.SERVING_HEADER_PATHS)
    assert {"rlk_mx4_quantize", "rlk_mx4_linear", "rlk_mx4_codes_bytes", "rlk_mx4_scales_bytes",
            "rlk_mx4_linear_workspace_bytes"} <= set(names)
    for n in names:
        assert hasattr(lib, n), n
        assert getattr(lib, n).argtypes is not None, n


def quant(x=P, n=4, d=64, ld=64, codes=2 * P, cb=1 << 20, scales=3 * P, sb=1 << 20, values=None, ldv=0):
    return rlk.load_library().rlk_mx4_quantize(x, n, d, ld, codes, cb, scales, sb, values, ldv, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL),
    (dict(x=P + 2), ALIGN), (dict(codes=P + 8), ALIGN), (dict(scales=P + 4), ALIGN),
    (dict(values=P + 8, ldv=64), ALIGN),
    (dict(n=-1), SHAPE), (dict(n=(1 << 22) + 1), SHAPE), (dict(d=48), SHAPE), (dict(d=0), SHAPE),
    (dict(d=65568, ld=65568), SHAPE), (dict(ld=56), SHAPE), (dict(ld=68), SHAPE), (dict(ld=1 << 62), SHAPE),
    (dict(values=4 * P, ldv=32), SHAPE), (dict(values=4 * P, ldv=68), SHAPE),
    (dict(cb=4095), WS), (dict(sb=255), WS),
])
def test_quantize_refuses(kw, code):
    assert quant(**kw) == code


def lin(h=P, n=4, d=64, ld=64, wc=2 * P, ws=3 * P, L=None, out=4 * P, work=5 * P, wb=1 << 20):
    L = L if L is not None else VocabLayout(1024, 1000, 1024, 8, 1)
    return rlk.load_library().rlk_mx4_linear(h, n, d, ld, wc, ws, ctypes.byref(L) if L is not False else None, out,
                                             work, wb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), NULL), (dict(wc=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL), (dict(work=None), NULL),
    (dict(L=False), NULL),
    (dict(h=P + 8), ALIGN), (dict(wc=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(work=P + 8), ALIGN),
    (dict(n=-1), SHAPE), (dict(d=33), SHAPE), (dict(ld=32), SHAPE), (dict(ld=66), SHAPE), (dict(ld=(1 << 21) + 8), SHAPE),
    (dict(L=VocabLayout(1000, 1000, 1024, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 0, 1024, 8, 1)), SHAPE),
    (dict(L=VocabLayout(1024, 1025, 1024, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 1000, 1020, 8, 1)), SHAPE),
    (dict(L=VocabLayout(1024, 1000, 1016, 8, 1)), SHAPE), (dict(L=VocabLayout(1024, 1000, 1024, 4, 1)), SHAPE),
    (dict(L=VocabLayout(1024, 1000, 1024, 8, 3)), GROUPS), (dict(wb=4096 + 255), WS),
])
def test_linear_refuses(kw, code):
    assert lin(**kw) == code


def test_no_rows_enqueue_nothing():
    assert quant(n=0, x=None, codes=None, scales=None, cb=0, sb=0) == OK
    assert lin(n=0, h=None, wc=None, ws=None, out=None, work=None, wb=0) == OK
    assert quant(n=0, d=48) == SHAPE


def test_binding_checks_tensors():
    assert rlk._bytes_tensor(torch.empty(100, dtype=torch.uint8, device=META), 100, META, "codes").numel() == 100
    for bad in (torch.empty(99, dtype=torch.uint8, device=META), torch.empty(100, dtype=torch.int8, device=META),
                torch.empty(100, dtype=torch.uint8), torch.empty(200, dtype=torch.uint8, device=META)[::2]):
        with pytest.raises(ValueError):
            rlk._bytes_tensor(bad, 100, META, "codes")
    with pytest.raises(ValueError):  # not on a device
        rlk.mx4_quantize(torch.zeros((4, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        rlk.mx4_linear(torch.zeros((4, 64), dtype=torch.bfloat16), None, None, vocab_real=10, vocab_padded=64)


def test_a_stream_of_another_device_is_refused():
    """Before anything is asked of the stream; a stream's device is all that is read."""
    class Stream:
        device = torch.device("cuda", 1)

    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=META)
    with pytest.raises(ValueError, match="stream is on cuda:1, x on meta"):
        rlk.mx4_quantize(x, stream=Stream())
    with pytest.raises(ValueError, match="stream is on cuda:1, x on meta"):
        rlk.mx4_quantize(x=x, stream=Stream())
    with pytest.raises(ValueError, match="hidden on meta"):
        rlk.mx4_linear(x, None, None, vocab_real=10, vocab_padded=64, stream=Stream())
    with pytest.raises(ValueError, match="logits on meta"):
        rlk.draft_verify(x, None, None, None, None, temperature=1.0, policy_logp=None, ref_logp=None, lse=None,
                         support_state=None, vocab_real=10, stream=Stream())
