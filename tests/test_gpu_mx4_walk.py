"""The wide 4-bit product where a workgroup takes two and more tiles of a d
above 256: the next tile's first half stages are loaded by the current one,
whose stores may still be in flight. Every logit against the exact sum: the
inputs' products are multiples of 1/4 and their sums stay below 2^24 quarters,
so float32 holds them in any order and the rounding to BF16 is the only one.
"""
import numpy as np
import pytest

import datagen
from oracle import mx4 as MX

from gpu_util import say
from test_gpu_mx4 import exact_matrix, run_linear

pytestmark = pytest.mark.gpu

# 256 workgroups: three to seven tiles each. d of two stages of 256 (both load from the next tile), three, four, five, nine;
# one band of rows and several; rows and columns that end inside a tile, so that waves go from whole tiles, whose stores
# stay in flight, to cut ones and back, and a batch whose rows end with a tile
SHAPES = [(1100, 512, 33001, 33024), (2100, 768, 20001, 20032), (1300, 1024, 30000, 30016), (600, 1056, 66001, 66048),
          (300, 544, 140001, 140032), (1024, 512, 40000, 40000), (1100, 2080, 33001, 33024), (200, 1312, 200001, 200064)]


@pytest.mark.parametrize("n,d,vr,vp", SHAPES)
def test_every_logit_of_many_tiles_is_exact(n, d, vr, vp):
    tiles = -(-n // 256) * -(-vp // 256)
    assert tiles > 2 * 256 and d > 256
    say(f"case: exact 4-bit linear {n} x {d} x {vr}/{vp}, {tiles} tiles")
    rng = np.random.default_rng(n + d + vr)
    hb, wb = exact_matrix(rng, n, d), exact_matrix(rng, vr, d)
    got = run_linear(hb, wb, vp)
    h, w = MX.decode_bf16(hb).astype(np.float32), MX.decode_bf16(wb).astype(np.float32)
    for at in range(0, n, 256):
        want = datagen.f32_to_bf16_bits(h[at:at + 256] @ w.T)
        same = np.array_equal(got[at:at + 256], want)
        assert same, (at, np.argwhere(got[at:at + 256] != want)[:4].tolist())
