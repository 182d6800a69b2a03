"""GPU parity of the microscaled 4-bit quantisation and LM-head product against
the float64 oracle (oracle/mx4.py).

Quantisation is exact: codes, scale bytes and values must equal the oracle's
byte for byte, the zeros of missing rows and values included. The product of
values whose partial sums are all exact in float32 must equal the rounded exact
sum bit for bit; with random values a logit is off by at most half a BF16 step
(2^-8 of the value) plus the float32 sum's error: d additions, each off by at
most 2^-23 of the sum of the magnitudes (a whole unit: the matrix cores' adders
inside one instruction are not specified to round to nearest).
"""
import numpy as np
import pytest

import datagen
import invariant_token_log_fp32_amd as rlk
from oracle import mx4 as MX

from gpu_util import say, to_host

pytestmark = pytest.mark.gpu


def upload(bits, cols=None):
    """Device copy of a BF16 matrix, with a row stride of ``cols`` (extra columns NaN)."""
    import torch
    n, d = bits.shape
    buf = np.full((n, cols or d), 0x7FC0, dtype=np.uint16)
    buf[:, :d] = bits
    return torch.from_numpy(buf.view(np.int16)).to("cuda:0").view(torch.bfloat16)[:, :d]


def random_bits(rng, n, d, spread=6):
    x = rng.normal(0, 1, (n, d)) * np.exp2(rng.integers(-spread, spread + 1, (n, -(-d // 32)))).repeat(32, 1)[:, :d]
    return datagen.f32_to_bf16_bits(x.astype(np.float32))


def check_quantize(bits, cols=None, vcols=None):
    import torch
    n, d = bits.shape
    x = upload(bits, cols)
    need = rlk.mx4_bytes(n, d)
    codes = torch.full((need[0] + 64,), 0xA5, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((need[1] + 64,), 0xA5, dtype=torch.uint8, device="cuda:0")
    values = torch.full((n + 1, vcols or d), 0x5A5A, dtype=torch.int16, device="cuda:0").view(torch.bfloat16)
    rlk.mx4_quantize(x, codes=codes, scales=scales, values_out=values[:n, :d])
    torch.cuda.synchronize()
    code, byte = MX.quantize(bits)
    want_c, want_s = MX.pack(code, byte)
    got_c, got_s = to_host(codes), to_host(scales)
    assert np.array_equal(got_s[:need[1]], want_s), "scale bytes differ"
    assert np.array_equal(got_c[:need[0]], want_c), "codes differ"
    assert (got_c[need[0]:] == 0xA5).all() and (got_s[need[1]:] == 0xA5).all(), "bytes behind the matrix were written"
    got_v = to_host(values.view(torch.int16)).view(np.uint16)
    want = MX.values(code, byte)
    want_v = np.where(np.isnan(want), 0x7FC0, (want.astype(np.float32).view(np.uint32) >> 16)).astype(np.uint16)
    assert np.array_equal(got_v[:n, :d], want_v), "values differ"
    assert (got_v[n:] == 0x5A5A).all() and (got_v[:, d:] == 0x5A5A).all(), "values were written behind the matrix"


@pytest.mark.parametrize("n,d,pad,vpad", [(1, 32, 0, 0), (33, 96, 8, 16), (8, 256, 0, 0), (31, 4096, 0, 0), (100, 2080, 96, 8),
                                          (257, 288, 0, 0), (64, 65536, 0, 0)])
def test_quantize_matches_the_oracle(n, d, pad, vpad):
    say(f"case: quantise {n} x {d}, stride + {pad}")
    check_quantize(random_bits(np.random.default_rng(n + d), n, d), d + pad, d + vpad)


def test_quantize_every_bf16_pattern():
    """Each of the 65536 patterns as the largest value of a block, alone and
    beside an eighth of itself, and beside a larger value that sets the scale."""
    say("case: quantise all 65536 BF16 patterns")
    every = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    blocks = np.zeros((65536, 32), np.uint16)
    blocks[:, 5] = every
    exponent = (every >> 7) & 0xFF
    blocks[:, 9] = np.where((exponent > 3) & (exponent < 255), every - (3 << 7), 0)
    blocks[:, 31] = np.where((exponent > 3) & (exponent < 255), (every ^ 0x8000) - (2 << 7), 0x8000)
    check_quantize(blocks.reshape(2048, 1024))
    other = np.zeros((65536, 32), np.uint16)
    other[:, 0] = np.where(exponent < 252, ((exponent + 2) << 7) | 0x7F, 0)   # the scale of a value up to 8 times larger
    other[:, 17] = every
    check_quantize(other.reshape(2048, 1024))


def test_quantize_in_place_and_on_another_stream():
    import torch
    say("case: quantise in place, side stream")
    bits = random_bits(np.random.default_rng(8), 70, 352)
    x = upload(bits, 360)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes, scales, values = rlk.mx4_quantize(x, values_out=x, return_values=True, stream=side)
    side.synchronize()
    code, byte = MX.quantize(bits)
    want_c, want_s = MX.pack(code, byte)
    assert values is x
    assert np.array_equal(to_host(codes), want_c) and np.array_equal(to_host(scales), want_s)
    got = to_host(x.float()).astype(np.float64)
    assert np.array_equal(got, MX.values(code, byte))


def exact_matrix(rng, n, d, density=1.0):
    """Grid values times 1 or 2 a block: every product is a multiple of 1/4 of
    magnitude up to 144, so sums of 16384 of them stay below 2^24 quarters."""
    v = rng.choice(MX.GRID, (n, d)) * rng.choice([-1.0, 1.0], (n, d)) * (rng.random((n, d)) < density)
    v[:, ::32] = 6.0 * rng.choice([-1.0, 1.0], (n, -(-d // 32)))   # the block's maximum: the scale is 2^0
    v = v * rng.choice([1.0, 2.0], (n, d // 32)).repeat(32, 1)
    return datagen.f32_to_bf16_bits(v.astype(np.float32))


def run_linear(hb, wb, vp, hpad=0, opad=0, **kw):
    import torch
    n, d = hb.shape
    vr = wb.shape[0]
    wc, ws = rlk.mx4_quantize(upload(wb))
    out = torch.full((n + 1, vp + opad), 0x5A5A, dtype=torch.int16, device="cuda:0").view(torch.bfloat16)
    rlk.mx4_linear(upload(hb, d + hpad), wc, ws, vocab_real=vr, vocab_padded=vp, out=out[:n], **kw)
    torch.cuda.synchronize()
    got = to_host(out.view(torch.int16)).view(np.uint16)
    assert (got[n:] == 0x5A5A).all() and (got[:, vp:] == 0x5A5A).all(), "logits were written behind the matrix"
    assert (got[:n, vr:vp] == 0xFF80).all(), "pad columns"
    return got[:n, :vr]


# below, at and above every border of rows (32 a tile; the wide kernel's 256), of columns and of d
SHAPES = [(1, 32, 1, 64), (1, 4096, 700, 768), (5, 96, 300, 320), (17, 256, 64, 64), (32, 288, 257, 320),
          (33, 512, 1999, 2048), (64, 1056, 1000, 1024), (65, 224, 511, 512), (96, 64, 129, 192), (127, 320, 300, 320),
          (128, 768, 1023, 1024), (129, 1024, 255, 256), (200, 544, 2049, 2112), (255, 256, 256, 256),
          (257, 448, 1999, 2048), (300, 2080, 900, 1024), (520, 32, 1300, 1344), (1100, 192, 14999, 15360),
          (2000, 256, 10000, 10240)]


@pytest.mark.parametrize("n,d,vr,vp", SHAPES)
def test_linear_is_exact_where_the_sums_are(n, d, vr, vp):
    say(f"case: exact 4-bit linear {n} x {d} x {vr}/{vp}")
    rng = np.random.default_rng(n * 7 + d)
    hb, wb = exact_matrix(rng, n, d), exact_matrix(rng, vr, d)
    got = run_linear(hb, wb, vp, hpad=8 * (n % 3), opad=8 * (d % 64 // 32))
    want = MX.decode_bf16(hb) @ MX.decode_bf16(wb).T
    assert np.array_equal(got, datagen.f32_to_bf16_bits(want.astype(np.float32)))


# every way of splitting d over the waves (1, 2, 4 and 8 parts; d above 4096 goes another way), for one, two and four
# blocks of rows, with more tiles of the vocabulary than teams of waves
SPLITS = [(3, 96, 70001, 70016), (20, 512, 70001, 70016), (32, 1024, 66001, 66048), (7, 1280, 35001, 35008),
          (1, 2304, 17001, 17024), (31, 4096, 16500, 16512), (1, 4352, 1000, 1024), (32, 8192, 500, 512),
          (40, 256, 66001, 66048), (64, 512, 66001, 66048), (33, 800, 33001, 33024), (50, 2048, 17001, 17024),
          (64, 2080, 9001, 9024), (48, 4096, 8300, 8320), (64, 5120, 600, 640),
          (70, 160, 33001, 33024), (128, 512, 33001, 33024), (100, 992, 33001, 33024), (65, 1056, 17001, 17024),
          (96, 3328, 8300, 8320), (128, 4096, 8300, 8320), (128, 4128, 300, 320), (130, 4352, 700, 704)]


@pytest.mark.parametrize("n,d,vr,vp", SPLITS)
def test_linear_is_exact_at_every_split_of_d(n, d, vr, vp):
    say(f"case: exact 4-bit linear {n} x {d} x {vr}/{vp}")
    rng = np.random.default_rng(n + 3 * d)
    hb, wb = exact_matrix(rng, n, d), exact_matrix(rng, vr, d)
    got = run_linear(hb, wb, vp)
    want = MX.decode_bf16(hb).astype(np.float32) @ MX.decode_bf16(wb).astype(np.float32).T   # exact in float32 in any order
    assert np.array_equal(got, datagen.f32_to_bf16_bits(want))


@pytest.mark.parametrize("n,d,vr,vp", [(3, 4096, 2000, 2048), (48, 1056, 3000, 3008), (300, 2080, 1500, 1536), (700, 512, 5000, 5056)])
def test_linear_random_values(n, d, vr, vp):
    say(f"case: random 4-bit linear {n} x {d} x {vr}/{vp}")
    rng = np.random.default_rng(n + d + vr)
    hb, wb = random_bits(rng, n, d, 2), random_bits(rng, vr, d, 2)
    got = MX.decode_bf16(run_linear(hb, wb, vp))
    want, total = MX.linear(hb, *MX.quantize(wb))
    off = np.abs(got - want)
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * d * 2.0 ** -23 * total
    assert (off <= tol).all(), float((off / tol).max())


def test_linear_rows_do_not_depend_on_the_batch():
    """The same rows in batches on both sides of every change of kernel, tile
    and row order: identical bytes."""
    import torch
    say("case: 4-bit linear, one row in many batches")
    rng = np.random.default_rng(21)
    n, d, vr, vp = 1030, 1312, 3001, 3008
    h, w = upload(random_bits(rng, n, d, 2)), upload(random_bits(rng, vr, d, 2))
    wc, ws = rlk.mx4_quantize(w)
    whole = to_host(rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp).view(torch.int16))
    for m in (1, 2, 16, 31, 33, 64, 65, 96, 128, 129, 192, 256, 257, 384, 512, 513, 1024):
        at = (n - m) // 2
        part = to_host(rlk.mx4_linear(h[at:at + m], wc, ws, vocab_real=vr, vocab_padded=vp).view(torch.int16))
        assert np.array_equal(part, whole[at:at + m]), m
    order = torch.from_numpy(rng.permutation(n)).to("cuda:0")
    mixed = to_host(rlk.mx4_linear(h[order].contiguous(), wc, ws, vocab_real=vr, vocab_padded=vp).view(torch.int16))
    assert np.array_equal(mixed, whole[to_host(order)])


@pytest.mark.parametrize("vr,vp", [(1001, 1024), (33000, 33024)])
def test_linear_rows_do_not_depend_on_the_batch_with_a_long_d(vr, vp):
    import torch
    say(f"case: 4-bit linear, d above 4096, {vr} columns, one row in several batches")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(22)
    n, d = 260, 4640
    h = torch.randn((n, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    wc, ws = rlk.mx4_quantize(torch.randn((vr, d), generator=gen, device="cuda:0").to(torch.bfloat16))
    whole = rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp)
    for m in (1, 32, 33, 128, 129):
        assert torch.equal(rlk.mx4_linear(h[9:9 + m], wc, ws, vocab_real=vr, vocab_padded=vp), whole[9:9 + m]), m


def test_offsets_past_31_bits():
    """A matrix of more than 2^32 bytes to quantise, logits of more than 2^31
    elements: the last rows as in a call of their own."""
    import torch
    say("case: 4-bit quantise 34000 x 65536, linear 14200 x 64 x 151936")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(1)
    n, d = 34000, 65536
    x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda:0")
    x[-40:] = torch.randn((40, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    c, s, v = rlk.mx4_quantize(x, return_values=True)
    c2, s2, v2 = rlk.mx4_quantize(x[-48:].contiguous(), return_values=True)   # 34000 - 48 is no multiple of 32: rows 16 ..
    assert torch.equal(v[-48:], v2)
    last = rlk.mx4_bytes(32, d)
    c3, s3 = rlk.mx4_quantize(x[-16:].contiguous())   # 34000 = 32 * 1062 + 16: the last tile's rows
    assert torch.equal(c[-last[0]:], c3) and torch.equal(s[-last[1]:], s3)
    del x, v, v2, c, c2
    n, d, vr, vp = 14200, 64, 151936, 152576
    h = torch.randn((n, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    w = torch.randn((vr, d), generator=gen, device="cuda:0").to(torch.bfloat16)
    wc, ws = rlk.mx4_quantize(w)
    out = rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp)
    tail = rlk.mx4_linear(h[-50:].contiguous(), wc, ws, vocab_real=vr, vocab_padded=vp)
    assert torch.equal(out[-50:], tail)


@pytest.mark.parametrize("n", [6, 300])
def test_linear_nan_and_infinite_rows(n):
    """NaN or an infinity in a hidden row makes that row NaN; in a projection
    row that column; nothing else changes."""
    say(f"case: 4-bit linear with NaN and infinities, {n} rows")
    rng = np.random.default_rng(5)
    d, vr, vp = 352, 500, 512
    hb, wb = exact_matrix(rng, n, d), exact_matrix(rng, vr, d)
    want = MX.decode_bf16(hb) @ MX.decode_bf16(wb).T
    hb[1, 40], hb[4, 351] = 0x7FC0, 0x7F80
    wb[7, 0], wb[499, 350] = 0xFF80, 0xFFC1
    got = MX.decode_bf16(run_linear(hb, wb, vp))
    bad = np.zeros(got.shape, bool)
    bad[[1, 4]] = True
    bad[:, [7, 499]] = True
    assert np.isnan(got[bad]).all()
    want_bits = datagen.f32_to_bf16_bits(want.astype(np.float32))
    assert np.array_equal(got[~bad], MX.decode_bf16(want_bits)[~bad])


def test_linear_graph_replays_match_eager():
    """Two captured graphs, each with its own workspace, replayed in turn with
    eager calls and new inputs between them."""
    import torch
    say("case: 4-bit quantise + linear in two graphs")
    rng = np.random.default_rng(6)
    d, vr, vp = 512, 3000, 3008
    w = upload(random_bits(rng, vr, d, 2))
    wc, ws = rlk.mx4_quantize(w)
    kept = []
    for n in (3, 290):
        h = upload(random_bits(rng, n, d, 2)).contiguous()
        out = torch.zeros((n, vp), dtype=torch.bfloat16, device="cuda:0")
        work = torch.zeros(rlk.mx4_linear_workspace_bytes(n, d), dtype=torch.uint8, device="cuda:0")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp, out=out, workspace=work)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rlk.mx4_quantize(w, codes=wc, scales=ws)
            rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp, out=out, workspace=work)
        kept.append((n, h, out, work, g))
    for again in range(4):
        for n, h, out, work, g in kept:
            h.copy_(upload(random_bits(rng, n, d, 2)))
            want = to_host(rlk.mx4_linear(h, wc, ws, vocab_real=vr, vocab_padded=vp).view(torch.int16))
            out.fill_(7.0)
            work.fill_(0x33)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(to_host(out.view(torch.int16)), want), (again, n)


def test_refusals_on_the_device():
    import torch
    x = torch.zeros((4, 48), dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(rlk.RlkError):   # d is not a multiple of 32
        rlk.mx4_quantize(x)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda:0")
    for kw in (dict(codes=torch.empty(10, dtype=torch.uint8, device="cuda:0")),
               dict(scales=torch.empty(10, dtype=torch.uint8, device="cuda:0")),
               dict(values_out=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda:0")),
               dict(values_out=torch.empty((3, 64), dtype=torch.bfloat16, device="cuda:0"))):
        with pytest.raises(ValueError):
            rlk.mx4_quantize(x, **kw)
    with pytest.raises(ValueError):
        rlk.mx4_quantize(x.float())
    with pytest.raises(ValueError):
        rlk.mx4_quantize(x.t())
    with pytest.raises(rlk.RlkError):   # a row of a strided view that is not 16-byte aligned
        rlk.mx4_quantize(torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda:0")[:, 4:68])
    wc, ws = rlk.mx4_quantize(x)
    for bad in (dict(vocab_real=40, vocab_padded=64), ):    # more rows than the codes hold
        with pytest.raises(ValueError):
            rlk.mx4_linear(x, wc, ws, **bad)
    with pytest.raises(rlk.RlkError):
        rlk.mx4_linear(x, wc, ws, vocab_real=4, vocab_padded=72)
    with pytest.raises(ValueError):
        rlk.mx4_linear(x, wc, ws, vocab_real=4, vocab_padded=64, out=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(ValueError):
        rlk.mx4_linear(x, wc, ws, vocab_real=4, vocab_padded=64, workspace=torch.empty(16, dtype=torch.uint8, device="cuda:0"))
    assert rlk.mx4_linear(x[:0], wc, ws, vocab_real=4, vocab_padded=64).shape == (0, 64)
