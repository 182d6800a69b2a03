// BF16 logits out of the 32 x 32 blocks that the matrix instructions leave in
// the accumulators (the vocabulary fragment as the first operand): rounding,
// the exchange that gives a lane 16 neighbouring columns, 16-byte stores with
// the pad columns set to -inf.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "logp_device.hpp"

namespace rlk {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values rounded to BF16 (nearest even) in one 32-bit word, low first.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// 8 BF16 logits (4 packed pairs) at column c of a row; pad columns -inf.
__device__ __forceinline__ void store8(int64_t vocab_real, uint16_t* __restrict__ dst, int64_t c, uint32_t w0,
                                       uint32_t w1, uint32_t w2, uint32_t w3) {
  if (c + 8 > vocab_real) {
    const uint32_t w[4] = {w0, w1, w2, w3};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = (c + 2 * k < vocab_real) ? (w[k] & 0xFFFFu) : 0xFF80u;
      const uint32_t hi = (c + 2 * k + 1 < vocab_real) ? (w[k] & 0xFFFF0000u) : 0xFF800000u;
      o[k] = lo | hi;
    }
    w0 = o[0];
    w1 = o[1];
    w2 = o[2];
    w3 = o[3];
  }
  *reinterpret_cast<u32x4*>(dst) = u32x4{w0, w1, w2, w3};
}

// The 16 BF16 logits of block (i, j) that lane l stores, as 8 packed words:
// lane l holds, for q = 0..3, columns 8q + 4h .. +3 (h = l/32) of row l%32; one
// exchange with lane l^32 gives it the 16 columns 16h .. +15. The exchange of a
// lower half's word for an upper half's is one instruction.
__device__ __forceinline__ void swap_halves(uint32_t& low, uint32_t& high) {
  // lanes 32..63 of `low` with lanes 0..31 of `high`
  const auto r = __builtin_amdgcn_permlane32_swap(low, high, false, false);
  low = r[0];
  high = r[1];
}

__device__ __forceinline__ void block_words(const f32x16& v, uint32_t (&w)[8]) {
  w[0] = pack_bf16(v[0], v[1]);    // q = 0: stays in h = 0, to the partner in h = 1
  w[1] = pack_bf16(v[2], v[3]);
  w[2] = pack_bf16(v[8], v[9]);    // q = 2
  w[3] = pack_bf16(v[10], v[11]);
  w[4] = pack_bf16(v[4], v[5]);    // q = 1
  w[5] = pack_bf16(v[6], v[7]);
  w[6] = pack_bf16(v[12], v[13]);  // q = 3
  w[7] = pack_bf16(v[14], v[15]);
  swap_halves(w[0], w[2]);
  swap_halves(w[1], w[3]);
  swap_halves(w[4], w[6]);
  swap_halves(w[5], w[7]);
}

}  // namespace rlk
