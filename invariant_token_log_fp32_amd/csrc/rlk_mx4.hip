// Microscaled 4-bit quantisation and the LM-head product with both operands in
// that form, and the C ABI declared in include/rlk_mx4.h.
//
// Kernels:
//   k_mx4_quantize   one wave per 8 rows x 256 values: 8 lanes read the 128
//                    bytes of two blocks of a row, four lanes hold a block,
//                    whose largest magnitude comes from packed 16-bit maxima
//                    and two steps over the four lanes; the hardware's
//                    conversion rounds to 4 bits (nearest even, saturating).
//   k_mx4_rows       a wave takes 32 rows x 64 vocabulary columns of the
//                    product and streams both operands from memory straight
//                    into the matrix instructions' registers: the packed
//                    layout holds, lane after lane, what one instruction takes.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "bf16_store.hpp"
#include "logp_device.hpp"
#include "rlk_logp.h"
#include "rlk_mx4.h"

namespace rlk_mx4 {

using rlk::f32x16;
using rlk::u32x4;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kTileRows = 32;        // rows of a packed tile: one operand of the 32x32x64 instruction
constexpr int kStepK = 64;           // values of a row in one instruction
constexpr int kStepBytes = 1024;     // codes of a tile's step: 64 lanes x 16 bytes
constexpr int kScaleK = 256;         // values of a row whose scale bytes fill one word a lane
constexpr int kScaleBytes = 256;     // scales of a tile's four steps: 64 lanes x 4 bytes
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxLd = int64_t(1) << 21;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int kMaxD = 65536;

static bool shape_ok(int64_t n_rows, int64_t d) {
  return n_rows >= 0 && n_rows <= kMaxRows && d >= 32 && d <= kMaxD && d % 32 == 0;
}
static int64_t row_tiles(int64_t n_rows) { return (n_rows + kTileRows - 1) / kTileRows; }
static int64_t scale_steps(int64_t d) { return (d + kScaleK - 1) / kScaleK; }

// ---------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------

constexpr int kQRows = 8;      // rows of a wave's tile
constexpr int kQThreads = 256;

// Largest of the two 16-bit halves of each word, over the word and the quad of lanes.
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("v_pk_max_u16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

template <int Ctrl>
__device__ __forceinline__ uint32_t quad_perm(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), Ctrl, 0xF, 0xF, true));
}

// Codes of 8 values (one lane's quarter of a block) and the block's scale byte.
__device__ __forceinline__ void quantize8(const u32x4& v, uint32_t& code, uint32_t& byte) {
  const uint32_t mask = 0x7FFF7FFFu;
  uint32_t m = pk_max_u16(pk_max_u16(v.x & mask, v.y & mask), pk_max_u16(v.z & mask, v.w & mask));
  m = pk_max_u16(m, quad_perm<0xB1>(m));  // lanes 1 0 3 2
  m = pk_max_u16(m, quad_perm<0x4E>(m));  // lanes 2 3 0 1
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
  const uint32_t top = lo > hi ? lo : hi;
  if (top >= 0x7F80u) {  // NaN or an infinity in the block
    byte = 255u;
    code = 0u;
    return;
  }
  // floor(log2 a) = exponent field - 127; a subnormal or zero field ends at byte 0 as well
  const uint32_t field = top >> 7;
  byte = field > 2u ? field - 2u : 0u;
  const float up = __uint_as_float((254u - byte) << 23);  // 2^-e, at most 2^127
  float x[8];
  rlk::unpack8(v, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * up;  // exact: below 8 in magnitude
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], 1.0f, 3);
  code = c;
}

// The BF16 values that 8 codes stand for.
__device__ __forceinline__ u32x4 dequantize8(uint32_t code, uint32_t byte) {
  if (byte == 255u) return u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  const float s = __uint_as_float(byte ? byte << 23 : 0x00400000u);  // 2^e; 2^-127 is subnormal
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
  const float x[8] = {a.x * s, a.y * s, b.x * s, b.y * s, c.x * s, c.y * s, d.x * s, d.y * s};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // exact in BF16: the low halves are zero
    w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xFFFF0000u);
  return u32x4{w[0], w[1], w[2], w[3]};
}

__global__ __launch_bounds__(kQThreads) void k_mx4_quantize(const uint16_t* x, int64_t n_rows, int d,
                                                            int64_t ldx, int steps4, int64_t n_work,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                            uint16_t* values, int64_t ldv) {  // values may be x
  const int lane = threadIdx.x & 63;
  const int64_t work = static_cast<int64_t>(blockIdx.x) * (kQThreads / 64) + (threadIdx.x >> 6);
  if (work >= n_work) return;
  const int64_t group = work / steps4;              // 8 rows
  const int s4 = static_cast<int>(work % steps4);   // 256 values
  const int64_t row = group * kQRows + (lane >> 3);
  const int k0 = s4 * kScaleK + (lane & 7) * 8;
  u32x4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = k0 + u * kStepK;
    v[u] = u32x4{0u, 0u, 0u, 0u};
    if (row < n_rows && k < d) v[u] = *reinterpret_cast<const u32x4*>(x + row * ldx + k);
  }
  const int64_t tile = row / kTileRows;
  const int r = static_cast<int>(row % kTileRows);
  const int h = (lane >> 2) & 1;
  uint32_t packed = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t code, byte;
    quantize8(v[u], code, byte);
    packed |= byte << (8 * u);
    const int64_t step = tile * (4 * steps4) + 4 * s4 + u;
    *reinterpret_cast<uint32_t*>(codes + step * kStepBytes + h * 512 + r * 16 + (lane & 3) * 4) = code;
    const int k = k0 + u * kStepK;
    if (values != nullptr && row < n_rows && k < d)
      *reinterpret_cast<u32x4*>(values + row * ldv + k) = dequantize8(code, byte);
  }
  if ((lane & 3) == 0)
    *reinterpret_cast<uint32_t*>(scales + (tile * steps4 + s4) * kScaleBytes + h * 128 + r * 4) = packed;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

struct Geo {
  const uint8_t* __restrict__ hc;  // codes and scales of the hidden states
  const uint8_t* __restrict__ hs;
  const uint8_t* __restrict__ wc;  // and of the projection
  const uint8_t* __restrict__ ws;
  int64_t n_rows;
  int64_t vocab_real;
  int64_t vocab_padded;
  int64_t ldo;
  int steps4;       // groups of four steps along d
};

template <int Sel>
__device__ __forceinline__ f32x16 mma(const i32x4& w, const i32x4& h, const f32x16& c, int sw, int sh) {
  const i32x8 a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b = __builtin_shufflevector(h, h, 0, 1, 2, 3, -1, -1, -1, -1);
  // 4: E2M1 for either operand; Sel: which byte of the scale words belongs to this step
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, Sel, sw, Sel, sh);
}

constexpr int kRowsThreads = 256;
constexpr int kRowsCols = 64;  // columns of a wave

__global__ __launch_bounds__(kRowsThreads) void k_mx4_rows(Geo g, int64_t col_tiles, int64_t n_work,
                                                           uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int64_t work = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 64) + (threadIdx.x >> 6);
  if (work >= n_work) return;
  const int64_t ct = work % col_tiles;
  const int64_t rt = work / col_tiles;
  const int64_t w_tiles = (g.vocab_real + kTileRows - 1) / kTileRows;
  const int64_t steps = 4 * static_cast<int64_t>(g.steps4);
  f32x16 acc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[j][e] = 0.0f;
  const int64_t t0 = 2 * ct, t1 = 2 * ct + 1;
  const int64_t wt[2] = {t0 < w_tiles ? t0 : w_tiles - 1, t1 < w_tiles ? t1 : w_tiles - 1};  // past the end: any tile, not stored
  const i32x4* hc = reinterpret_cast<const i32x4*>(g.hc + rt * steps * kStepBytes) + lane;
  const int* hs = reinterpret_cast<const int*>(g.hs + rt * g.steps4 * kScaleBytes) + lane;
  const i32x4* wc[2];
  const int* ws[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    wc[j] = reinterpret_cast<const i32x4*>(g.wc + wt[j] * steps * kStepBytes) + lane;
    ws[j] = reinterpret_cast<const int*>(g.ws + wt[j] * g.steps4 * kScaleBytes) + lane;
  }
  for (int s4 = 0; s4 < g.steps4; ++s4) {
    const int sh = hs[s4 * 64];
    const int sw[2] = {ws[0][s4 * 64], ws[1][s4 * 64]};
    i32x4 h[4], w[2][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      h[u] = hc[(4 * s4 + u) * 64];
#pragma unroll
      for (int j = 0; j < 2; ++j) w[j][u] = wc[j][(4 * s4 + u) * 64];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      acc[j] = mma<0>(w[j][0], h[0], acc[j], sw[j], sh);
      acc[j] = mma<1>(w[j][1], h[1], acc[j], sw[j], sh);
      acc[j] = mma<2>(w[j][2], h[2], acc[j], sw[j], sh);
      acc[j] = mma<3>(w[j][3], h[3], acc[j], sw[j], sh);
    }
  }
  const int h = lane >> 5;
  const int64_t row = rt * kTileRows + (lane & 31);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t w[8];
    rlk::block_words(acc[j], h, w);
    const int64_t c = (2 * ct + j) * kTileRows + 16 * h;
    if (row < g.n_rows && c < g.vocab_padded) {
      rlk::store8(g.vocab_real, out + row * g.ldo + c, c, w[0], w[1], w[2], w[3]);
      rlk::store8(g.vocab_real, out + row * g.ldo + c + 8, c + 8, w[4], w[5], w[6], w[7]);
    }
  }
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static int32_t launched() { return hipGetLastError() == hipSuccess ? RLK_OK : RLK_ERR_HIP; }

static int32_t launch_quantize(const uint16_t* x, int64_t n_rows, int64_t d, int64_t ldx, uint8_t* codes,
                               uint8_t* scales, uint16_t* values, int64_t ldv, hipStream_t stream) {
  const int64_t steps4 = scale_steps(d);
  const int64_t n_work = row_tiles(n_rows) * (kTileRows / kQRows) * steps4;  // below 2^19 * 2^8
  const int64_t blocks = (n_work + kQThreads / 64 - 1) / (kQThreads / 64);
  k_mx4_quantize<<<dim3(static_cast<unsigned>(blocks)), dim3(kQThreads), 0, stream>>>(
      x, n_rows, static_cast<int>(d), ldx, static_cast<int>(steps4), n_work, codes, scales, values, ldv);
  return launched();
}

static int32_t check_layout(const rlk_vocab_layout* L) {
  if (L == nullptr) return RLK_ERR_NULL;
  if (L->n_shards != 8) return RLK_ERR_SHAPE;
  if (L->vocab_padded < 64 || L->vocab_padded > kMaxVocab || L->vocab_padded % 64 != 0) return RLK_ERR_SHAPE;
  if (L->vocab_real < 1 || L->vocab_real > L->vocab_padded || L->vocab_real > kMaxRows) return RLK_ERR_SHAPE;
  if (L->row_stride < L->vocab_padded || L->row_stride % 8 != 0) return RLK_ERR_SHAPE;
  if (!(L->groups == 1 || L->groups == 2 || L->groups == 4 || L->groups == 8)) return RLK_ERR_GROUPS;
  return RLK_OK;
}

}  // namespace rlk_mx4

extern "C" {

size_t rlk_mx4_codes_bytes(int64_t n_rows, int64_t d) {
  using namespace rlk_mx4;
  if (!shape_ok(n_rows, d)) return 0;
  return static_cast<size_t>(row_tiles(n_rows) * scale_steps(d)) * 4 * kStepBytes;
}

size_t rlk_mx4_scales_bytes(int64_t n_rows, int64_t d) {
  using namespace rlk_mx4;
  if (!shape_ok(n_rows, d)) return 0;
  return static_cast<size_t>(row_tiles(n_rows) * scale_steps(d)) * kScaleBytes;
}

int32_t rlk_mx4_quantize(const uint16_t* x, int64_t n_rows, int64_t d, int64_t row_stride,
                         uint8_t* codes, size_t codes_bytes, uint8_t* scales, size_t scales_bytes,
                         uint16_t* values_out, int64_t values_stride, hipStream_t stream) {
  using namespace rlk_mx4;
  if (!shape_ok(n_rows, d)) return RLK_ERR_SHAPE;
  if (row_stride < d || row_stride % 8 != 0) return RLK_ERR_SHAPE;
  if (n_rows > 0 && row_stride > INT64_MAX / 2 / n_rows) return RLK_ERR_SHAPE;
  if (values_out != nullptr) {
    if (values_stride < d || values_stride % 8 != 0) return RLK_ERR_SHAPE;
    if (n_rows > 0 && values_stride > INT64_MAX / 2 / n_rows) return RLK_ERR_SHAPE;
  }
  if (n_rows == 0) return RLK_OK;
  if (!x || !codes || !scales) return RLK_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16) || (values_out && !aligned(values_out, 16)))
    return RLK_ERR_ALIGN;
  if (codes_bytes < rlk_mx4_codes_bytes(n_rows, d) || scales_bytes < rlk_mx4_scales_bytes(n_rows, d))
    return RLK_ERR_WORKSPACE;
  return launch_quantize(x, n_rows, d, row_stride, codes, scales, values_out, values_stride, stream);
}

size_t rlk_mx4_linear_workspace_bytes(int64_t n_rows, int64_t d_model) {
  return rlk_mx4_codes_bytes(n_rows, d_model) + rlk_mx4_scales_bytes(n_rows, d_model);
}

int32_t rlk_mx4_linear(const uint16_t* hidden, int64_t n_rows, int64_t d_model, int64_t hidden_stride,
                       const uint8_t* weight_codes, const uint8_t* weight_scales, const rlk_vocab_layout* layout,
                       uint16_t* logits_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace rlk_mx4;
  int32_t st = check_layout(layout);
  if (st != RLK_OK) return st;
  if (!shape_ok(n_rows, d_model)) return RLK_ERR_SHAPE;
  if (hidden_stride < d_model || hidden_stride % 8 != 0 || hidden_stride > kMaxLd) return RLK_ERR_SHAPE;
  if (n_rows > 0 && layout->row_stride > INT64_MAX / 2 / n_rows) return RLK_ERR_SHAPE;
  if (n_rows == 0) return RLK_OK;
  if (!hidden || !weight_codes || !weight_scales || !logits_out || !workspace) return RLK_ERR_NULL;
  if (!aligned(hidden, 16) || !aligned(weight_codes, 16) || !aligned(weight_scales, 16) || !aligned(logits_out, 16) ||
      !aligned(workspace, 16))
    return RLK_ERR_ALIGN;
  if (workspace_bytes < rlk_mx4_linear_workspace_bytes(n_rows, d_model)) return RLK_ERR_WORKSPACE;
  uint8_t* hc = static_cast<uint8_t*>(workspace);
  uint8_t* hs = hc + rlk_mx4_codes_bytes(n_rows, d_model);
  if ((st = launch_quantize(hidden, n_rows, d_model, hidden_stride, hc, hs, nullptr, 0, stream)) != RLK_OK) return st;
  Geo g;
  g.hc = hc;
  g.hs = hs;
  g.wc = weight_codes;
  g.ws = weight_scales;
  g.n_rows = n_rows;
  g.vocab_real = layout->vocab_real;
  g.vocab_padded = layout->vocab_padded;
  g.ldo = layout->row_stride;
  g.steps4 = static_cast<int>(scale_steps(d_model));
  const int64_t col_tiles = layout->vocab_padded / kRowsCols;
  const int64_t n_work = col_tiles * row_tiles(n_rows);
  const int64_t blocks = (n_work + kRowsThreads / 64 - 1) / (kRowsThreads / 64);
  if (blocks > INT32_MAX) return RLK_ERR_SHAPE;
  k_mx4_rows<<<dim3(static_cast<unsigned>(blocks)), dim3(kRowsThreads), 0, stream>>>(g, col_tiles, n_work, logits_out);
  return launched();
}

}  // extern "C"
