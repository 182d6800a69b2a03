// Microscaled 4-bit quantisation and the LM-head product with both operands in
// that form, and the C ABI declared in include/rlk_mx4.h.
//
// Kernels:
//   k_mx4_quantize   one wave per 8 rows x 256 values: 8 lanes read the 128
//                    bytes of two blocks of a row, four lanes hold a block,
//                    whose largest magnitude comes from packed 16-bit maxima
//                    and two steps over the four lanes; the hardware's
//                    conversion rounds to 4 bits (nearest even, saturating).
//                    Bound by memory: 151936 x 4096 with values 2.8 GB in 0.49
//                    to 0.52 ms, 5.4 to 5.7 TB/s (a large copy 4.8-5.1), codes
//                    and scales alone 1.6 GB in 0.29 ms.
//   k_mx4_stream     up to 128 rows, d up to 4096: the projection streamed past
//                    hidden states in registers. Bound by reading it: 332 MB of
//                    the 151936 x 4096 head, 1 row 59 us (5.6 TB/s; a bare read
//                    of as much takes 49 us), 48 rows 70 us, 128 rows 85 us.
//   k_mx4_tiles      more rows, and 33 to 128 rows of a longer d where the
//                    vocabulary fills half the GPU with its tiles: 256 x 256
//                    tiles, operands through LDS. 8192 rows of the head 2.42
//                    to 2.57 ms, 4.0 to 4.2 PFLOP/s: the bare scaled matrix
//                    instructions run at 6.3 on all compute units, where power
//                    holds the clock at 1.5 GHz.
//   k_mx4_rows       up to 32 rows of a longer d, up to 128 of a smaller
//                    vocabulary: a wave takes 32 rows x 64 vocabulary columns
//                    and streams both operands from memory straight into the
//                    matrix instructions' registers: the packed layout holds,
//                    lane after lane, what one takes. 1 row of 151936 x 8192
//                    121 us, 32 rows 127 us (661 MB, 5.2 to 5.5 TB/s).
// All of them add a logit's products in the same order (64 values of d an
// instruction, the accumulator carried), so its bits do not depend on the kernel.
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
__host__ __device__ static inline int64_t row_tiles(int64_t n_rows) { return (n_rows + kTileRows - 1) / kTileRows; }
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

// Scale byte of a block whose largest magnitude pattern is `top`: 255 where it
// holds NaN or an infinity, else floor(log2 a) - 2 + 127, at least 0 (the
// exponent field is floor(log2 a) + 127; a subnormal or zero one ends at 0 too).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t field = top >> 7;
  return top >= 0x7F80u ? 255u : (field > 2u ? field - 2u : 0u);
}

// Codes of 8 values of a block with that scale byte.
__device__ __forceinline__ uint32_t codes8(const u32x4& v, uint32_t byte) {
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
  return byte == 255u ? 0u : c;
}

// The same for one lane's quarter of a block, whose maximum the quad shares.
__device__ __forceinline__ void quantize8(const u32x4& v, uint32_t& code, uint32_t& byte) {
  const uint32_t mask = 0x7FFF7FFFu;
  uint32_t m = pk_max_u16(pk_max_u16(v.x & mask, v.y & mask), pk_max_u16(v.z & mask, v.w & mask));
  m = pk_max_u16(m, quad_perm<0xB1>(m));  // lanes 1 0 3 2
  m = pk_max_u16(m, quad_perm<0x4E>(m));  // lanes 2 3 0 1
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
  byte = scale_byte(lo > hi ? lo : hi);
  code = codes8(v, byte);
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

typedef i32x4 Frag4;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kSteps = kScaleK / kStepK;  // 4 instructions deep: one word of scales
constexpr int kRsrcWord3 = 0x00020000;    // raw buffer, 32-bit data format, no swizzle
constexpr int kNoLoad = 0x40000000;       // an offset behind the end of every resource

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6); }

// The 16 bytes of this lane in the KiB at byte `at` of a resource. The
// projection is read once: non-temporal (1 row of the 151936 x 4096 head: 62.6
// instead of 68.9 us).
constexpr int kNonTemporal = 2;
__device__ __forceinline__ Frag4 load_frag(__amdgpu_buffer_rsrc_t r, int lane, int at) {
  return __builtin_bit_cast(Frag4, __builtin_amdgcn_raw_buffer_load_b128(r, lane * 16, at, kNonTemporal));
}
__device__ __forceinline__ int load_word(__amdgpu_buffer_rsrc_t r, int lane, int at) {
  return static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(r, lane * 4, at, kNonTemporal));
}

// One step of a wave's tile against NB blocks of hidden rows.
template <int Sel, int NB>
__device__ __forceinline__ void stream_step(const Frag4& w, const Frag4 (&h)[NB], f32x16 (&acc)[NB], int sw,
                                            const int (&sh)[NB]) {
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = mma<Sel>(w, h[b], acc[b], sw, sh[b]);
}

constexpr int kRowsThreads = 256;
constexpr int kRowsCols = 64;  // columns of a wave
// Up to 128 rows with d above 4096 (where k_mx4_stream ends) run on
// k_mx4_rows if they are one block of 32, or if the vocabulary has fewer than
// 128 tiles of the wide kernel (half the compute units): 151936 x 8192, 32 rows
// 131 us (wide 183), 64 rows 225 (wide 188 to 197); 20000 x 16384, 64 rows 71 us (wide 113).
constexpr int64_t kRowsMost = 128;
constexpr int64_t kRowsTiles = 128;

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
    rlk::block_words(acc[j], w);
    const int64_t c = (2 * ct + j) * kTileRows + 16 * h;
    if (row < g.n_rows && c < g.vocab_padded) {
      rlk::store8(g.vocab_real, out + row * g.ldo + c, c, w[0], w[1], w[2], w[3]);
      rlk::store8(g.vocab_real, out + row * g.ldo + c + 8, c + 8, w[4], w[5], w[6], w[7]);
    }
  }
}

// ---------------------------------------------------------------------------
// product, up to 128 rows: the projection streamed past the hidden states
// ---------------------------------------------------------------------------

// Few rows are bound by reading the projection once. SP waves (1, 2, 4 or 8: as
// few as hold it) split d and keep their parts of the hidden states in registers
// for good; packed tiles of 32 vocabulary rows stream through: the first wave
// multiplies its part of a tile and hands the accumulators to the second in LDS
// while it begins the next tile, and so on, so every logit's sum still runs in
// increasing k. A fragment's registers take a later tile's as soon as it is
// multiplied, so loads are always on their way. (With d always in four parts a
// short d spends its time on turns: 77 x 1056 x 50021 21.7 us.)
constexpr int kStreamBlocks = 4;    // blocks of 32 hidden rows, at most
// Groups of 256 values of d, at most (d <= 4096): where the registers of four
// blocks of rows end (a wave's four groups take 256 for the hidden states, 64 for
// the projection and 64 for accumulators, of 512). One and two blocks would have
// room for more; they end here too, and what a longer d would gain was not measured.
constexpr int kStreamSteps4 = 16;

// Waves of a workgroup, workgroups of a compute unit, groups of 256 values that
// a wave holds at most and tiles that its registers hold ahead, by blocks of
// rows (NB) and groups (GP): what the 512 registers that the waves of a SIMD
// share allow, with 8 waves a compute unit for one and two blocks (48 rows of
// the 151936 x 4096 head: 70 us, with 4 waves 78 us).
constexpr int stream_waves(int nb) { return nb == 2 ? 8 : 4; }
constexpr int stream_groups(int nb) { return nb == 1 ? 2 : 1; }
constexpr int stream_most(int nb) { return nb == 2 ? 2 : 4; }
constexpr int stream_depth(int nb, int gp) { return (nb == 1 || nb == 4) && gp == 4 ? 1 : 2; }

// One lane's block of 32 values (64 bytes of BF16), quantised as k_mx4_quantize does.
__device__ __forceinline__ Frag4 quantize32(const u32x4 (&v)[4], uint32_t& byte) {
  const uint32_t mask = 0x7FFF7FFFu;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = pk_max_u16(m, pk_max_u16(pk_max_u16(v[i].x & mask, v[i].y & mask), pk_max_u16(v[i].z & mask, v[i].w & mask)));
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
  byte = scale_byte(lo > hi ? lo : hi);
  Frag4 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = static_cast<int>(codes8(v[i], byte));
  return f;
}

__device__ __forceinline__ void stream_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int GP>
struct StreamPart {     // a wave's part of a tile of the projection
  Frag4 f[GP * kSteps];
  int sc[GP];
};

template <int NB, int GP, int SP>
__global__ __launch_bounds__(stream_waves(NB) * 64, stream_waves(NB) * stream_groups(NB) / 4) void k_mx4_stream(
    Geo g, const uint16_t* __restrict__ hidden, int64_t ldh, int d, int tiles, int w_tiles, uint16_t* __restrict__ out) {
  constexpr int kDepth = stream_depth(NB, GP);
  constexpr int kTeams = stream_waves(NB) / SP;   // teams of SP waves, each with tiles of its own
  __shared__ f32x4 slots[kTeams][SP > 1 ? SP - 1 : 1][SP > 1 ? NB : 1][4][64];
  const int lane = threadIdx.x & 63;
  const int team = wave_id() / SP;
  const int w = wave_id() % SP;                   // this wave's place in its team
  const int per = (g.steps4 + SP - 1) / SP;       // groups of a wave, at most GP
  const int g0 = w * per;
  const int cnt = g.steps4 - g0 < per ? g.steps4 - g0 : per;  // may be below 1
  // this team's tiles: neighbours, so that the two halves of a line of logits meet in L2
  const int teams = static_cast<int>(gridDim.x) * kTeams;
  const int share = (tiles + teams - 1) / teams;
  const int first = (static_cast<int>(blockIdx.x) * kTeams + team) * share;
  const int n_tiles = tiles - first < share ? tiles - first : share;  // may be below 1
  const int64_t codes = static_cast<int64_t>(g.steps4) * (kSteps * kStepBytes);  // of a packed tile
  const int64_t scales = static_cast<int64_t>(g.steps4) * kScaleBytes;

  // this wave's part of the i-th tile; behind the last one nothing is fetched
  const auto rsrcs = [&](int i, __amdgpu_buffer_rsrc_t& rc, __amdgpu_buffer_rsrc_t& rs) {
    const int t = first + i < w_tiles ? first + i : w_tiles - 1;  // pad columns alone: any tile, not stored
    const int most = i < n_tiles ? kNoLoad : 0;
    rc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(g.wc + t * codes + static_cast<int64_t>(g0) * (kSteps * kStepBytes)), 0, most, kRsrcWord3);
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.ws + t * scales + static_cast<int64_t>(g0) * kScaleBytes), 0,
                                           most, kRsrcWord3);
  };
  StreamPart<GP> part[kDepth];
#pragma unroll
  for (int p = 0; p < kDepth; ++p) {
    __amdgpu_buffer_rsrc_t rc, rs;
    rsrcs(p, rc, rs);
#pragma unroll
    for (int q = 0; q < GP; ++q)
      if (q < cnt) {
        part[p].sc[q] = load_word(rs, lane, q * kScaleBytes);
#pragma unroll
        for (int u = 0; u < kSteps; ++u) part[p].f[q * kSteps + u] = load_frag(rc, lane, (q * kSteps + u) * kStepBytes);
      }
  }

  Frag4 hf[GP * kSteps][NB];
  int hsc[GP][NB];
#pragma unroll
  for (int q = 0; q < GP; ++q) {
    if (q >= cnt) continue;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (NB == 1) {
        // few enough rows for every workgroup to quantise them itself: no launch before this one
        const int row = lane & 31;
        uint32_t word = 0;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int k = (g0 + q) * kScaleK + u * kStepK + (lane >> 5) * 32;
          u32x4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = u32x4{0u, 0u, 0u, 0u};
            if (row < g.n_rows && k < d) v[i] = *reinterpret_cast<const u32x4*>(hidden + row * ldh + k + 8 * i);
          }
          uint32_t byte;
          hf[q * kSteps + u][b] = quantize32(v, byte);
          word |= byte << (8 * u);
        }
        hsc[q][b] = static_cast<int>(word);
      } else {
        const int t = b < row_tiles(g.n_rows) ? b : 0;  // (three blocks of rows run as four)
        const uint8_t* at = g.hc + t * codes + static_cast<int64_t>(g0 + q) * (kSteps * kStepBytes);
#pragma unroll
        for (int u = 0; u < kSteps; ++u) hf[q * kSteps + u][b] = *reinterpret_cast<const Frag4*>(at + u * kStepBytes + lane * 16);
        hsc[q][b] = *reinterpret_cast<const int*>(g.hs + t * scales + static_cast<int64_t>(g0 + q) * kScaleBytes + lane * 4);
      }
    }
  }

  // the i-th tile: its products, each fragment's registers then taking tile i + kDepth's
  const auto multiply = [&](StreamPart<GP>& p, int i, f32x16 (&acc)[NB]) {
    __amdgpu_buffer_rsrc_t rc, rs;
    rsrcs(i + kDepth, rc, rs);
#pragma unroll
    for (int q = 0; q < GP; ++q) {
      if (q >= cnt) continue;
      const int sw = p.sc[q];
      p.sc[q] = load_word(rs, lane, q * kScaleBytes);
      Frag4(&f)[GP * kSteps] = p.f;
      stream_step<0, NB>(f[q * kSteps], hf[q * kSteps], acc, sw, hsc[q]);
      f[q * kSteps] = load_frag(rc, lane, q * kSteps * kStepBytes);
      stream_step<1, NB>(f[q * kSteps + 1], hf[q * kSteps + 1], acc, sw, hsc[q]);
      f[q * kSteps + 1] = load_frag(rc, lane, (q * kSteps + 1) * kStepBytes);
      stream_step<2, NB>(f[q * kSteps + 2], hf[q * kSteps + 2], acc, sw, hsc[q]);
      f[q * kSteps + 2] = load_frag(rc, lane, (q * kSteps + 2) * kStepBytes);
      stream_step<3, NB>(f[q * kSteps + 3], hf[q * kSteps + 3], acc, sw, hsc[q]);
      f[q * kSteps + 3] = load_frag(rc, lane, (q * kSteps + 3) * kStepBytes);
    }
  };

  for (int turn = 0; turn < share + SP - 1; ++turn) {  // as many in every team: their barriers are one
    const int i = turn - w;
    const bool on = i >= 0 && i < n_tiles;  // uniform across the wave
    f32x16 acc[NB];
    if (on) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
          if (SP > 1 && w > 0) v = slots[team][w - 1][SP > 1 ? b : 0][e][lane];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[b][4 * e + k] = v[k];
        }
    }
    if (SP > 1) stream_barrier();  // every slot is read
    if (on) {
      if (kDepth == 1 || (i & 1) == 0)
        multiply(part[0], i, acc);
      else
        multiply(part[kDepth - 1], i, acc);
      if (SP > 1 && w < SP - 1) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            slots[team][SP > 1 ? w : 0][SP > 1 ? b : 0][e][lane] = f32x4{acc[b][4 * e], acc[b][4 * e + 1], acc[b][4 * e + 2], acc[b][4 * e + 3]};
      } else {
        const int h = lane >> 5;
        const int64_t c = static_cast<int64_t>(first + i) * kTileRows + 16 * h;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t x[8];
          rlk::block_words(acc[b], x);
          const int64_t row = b * kTileRows + (lane & 31);
          if (row < g.n_rows && c < g.vocab_padded) {
            rlk::store8(g.vocab_real, out + row * g.ldo + c, c, x[0], x[1], x[2], x[3]);
            rlk::store8(g.vocab_real, out + row * g.ldo + c + 8, c + 8, x[4], x[5], x[6], x[7]);
          }
        }
      }
    }
    if (SP > 1) stream_barrier();  // every slot is written
  }
}

// ---------------------------------------------------------------------------
// product, many rows: 256 x 256 tiles
// ---------------------------------------------------------------------------

constexpr int BM = 256;                   // rows of a workgroup's tile
constexpr int BN = 256;                   // vocabulary columns of it
constexpr int kTilesThreads = 256;        // 4 waves, 2 x 2, each 128 x 128
constexpr int kPanelTiles = BM / kTileRows;      // 8 packed tiles of either operand
constexpr int kMB = 4;                    // 32 x 32 blocks of a wave, either way
constexpr int kNB = 4;
constexpr int kHalfSteps = kSteps / 2;    // steps of a half stage (128 values of d)
constexpr int kHalfPanel = kPanelTiles * kHalfSteps * kStepBytes;  // 16 KB of codes of one operand
constexpr int kHalfBytes = 2 * kHalfPanel;                         // both operands
constexpr int kPanelScales = kPanelTiles * kScaleBytes;            // 2 KB of scales of one operand and stage
constexpr int kOffScales = 4 * kHalfBytes;                         // four half stages of codes, then two of scales
constexpr int kStageScales = 2 * kPanelScales;
constexpr int kSmemBytes = kOffScales + 2 * kStageScales;          // 136 KB
constexpr int kXcds = 8;
constexpr int kGroup = 32;                // tiles that an XCD's compute units take together
static_assert(BM == BN, "one panel shape for both operands");

typedef __attribute__((address_space(3))) void* LdsPtr;
typedef Frag4 Frag;

struct TileGeo {
  Geo g;
  int m_tiles;
  int n_tiles;
  int band;          // rows of tiles in a band (the last may have fewer)
  int chunk;         // columns of tiles in a chunk (8; with one band all of them)
  int64_t h_end;     // packed tiles of either operand
  int64_t w_end;
};

// The tiles of a workgroup. In order: chunks of columns of tiles, in a chunk
// bands of up to 4 rows, in a band rows fastest. Workgroup b runs on XCD b % 8,
// and an XCD's 32 workgroups take 32 neighbours of that order at a time (4 x 8
// tiles), which stream the same 12 panels through its L2, while the XCDs
// together go over one part of the projection for all rows. 256 tiles a round,
// no gaps. (Band after band, each over the whole projection: 2.51 instead of
// 2.44 ms for 8192 rows of the 151936 x 4096 head.)
struct Walk {
  int left;          // place in the chunk
  int col0;          // the chunk's first column of tiles
  int m_t, n_t;      // the tile

  __device__ __forceinline__ explicit Walk(const TileGeo& g) {
    left = (blockIdx.x % kXcds) * kGroup + blockIdx.x / kXcds;
    col0 = 0;
  }

  __device__ __forceinline__ void step() { left += kXcds * kGroup; }

  __device__ __forceinline__ bool find(const TileGeo& g) {
    while (col0 < g.n_tiles) {
      const int width = g.n_tiles - col0 < g.chunk ? g.n_tiles - col0 : g.chunk;
      if (left < g.m_tiles * width) {
        const int row0 = left / (g.band * width) * g.band;
        const int rest = left - row0 * width;
        const int rows = g.m_tiles - row0 < g.band ? g.m_tiles - row0 : g.band;
        m_t = row0 + rest % rows;
        n_t = col0 + rest / rows;
        return true;
      }
      left -= g.m_tiles * width;
      col0 += g.chunk;
    }
    return false;
  }
};

// What this wave loads of a tile: packed tiles 2w and 2w + 1 of either operand's
// 8, and the scales of four (waves 0 and 1 the hidden states', 2 and 3 the
// projection's). A tile behind the operand's end is replaced by its last one
// (its rows or columns are not stored), so every load is in range.
struct Tile {
  const uint8_t* h;      // the panels' first tiles
  const uint8_t* w;
  const uint8_t* scales; // of this wave's scales
  int h_at[2];           // byte offsets of this wave's tiles in them
  int w_at[2];
  int scales_at;         // and of this lane's (16 lanes a tile)
};

__device__ __forceinline__ Tile make_tile(const TileGeo& g, const Walk& at) {
  const int lane = threadIdx.x & 63;
  const int w = wave_id();
  const int codes = g.g.steps4 * (kSteps * kStepBytes), scales = g.g.steps4 * kScaleBytes;  // of a packed tile
  const int64_t h0 = static_cast<int64_t>(at.m_t) * kPanelTiles;
  int64_t w0 = static_cast<int64_t>(at.n_t) * kPanelTiles;
  if (w0 >= g.w_end) w0 = g.w_end - 1;  // pad columns alone
  const int64_t hl = g.h_end - h0, wl = g.w_end - w0;
  const int hn = static_cast<int>(hl < kPanelTiles ? hl : kPanelTiles) - 1;  // last tile of the panels
  const int wn = static_cast<int>(wl < kPanelTiles ? wl : kPanelTiles) - 1;
  Tile t;
  t.h = g.g.hc + h0 * codes;
  t.w = g.g.wc + w0 * codes;
  t.scales = w < 2 ? g.g.hs + h0 * scales : g.g.ws + w0 * scales;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t.h_at[i] = (2 * w + i < hn ? 2 * w + i : hn) * codes;
    t.w_at[i] = (2 * w + i < wn ? 2 * w + i : wn) * codes;
  }
  const int mine = (w & 1) * 4 + (lane >> 4), last = w < 2 ? hn : wn;
  t.scales_at = (mine < last ? mine : last) * scales + (lane & 15) * 16;
  return t;
}

// Every offset into a panel is below 2^23, kNoLoad is behind the resource's end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t panel_rsrc(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, kNoLoad, kRsrcWord3);
}

// Load i (0..3) of this wave's 4 KB of one operand's half stage: step i % 2 of
// its tile i / 2, lane after lane as it lies in memory. `half` counts half
// stages along d; below 0: an offset behind the resource's end, which fetches
// nothing (zeros), without a branch.
__device__ __forceinline__ void load_codes(const uint8_t* p, const int (&at)[2], int half, uint8_t* __restrict__ panel,
                                           int i) {
  const int lane = threadIdx.x & 63;
  const int off = at[i >> 1] + (half < 0 ? 0 : half) * (kHalfSteps * kStepBytes) + (i & 1) * kStepBytes;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(panel_rsrc(p), (LdsPtr)(panel + (4 * wave_id() + i) * kStepBytes), 16,
                                           lane * 16 + (half < 0 ? kNoLoad : 0), off, 0, 0);
}

// The scales of a stage, four tiles of one panel in a wave's one load.
__device__ __forceinline__ void load_scales(const Tile& t, int kt, uint8_t* __restrict__ scales) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(panel_rsrc(t.scales), (LdsPtr)(scales + wave_id() * 4 * kScaleBytes), 16,
                                           t.scales_at + (kt < 0 ? kNoLoad : 0), (kt < 0 ? 0 : kt) * kScaleBytes, 0, 0);
}

// Half stage `half` (of stage half / 2) into its LDS buffer; the first half of
// a stage brings the stage's scales.
__device__ __forceinline__ void load_half(const Tile& t, int half, int buf, uint8_t* __restrict__ smem) {
  if ((buf & 1) == 0) load_scales(t, half < 0 ? -1 : half >> 1, smem + kOffScales + (buf >> 1) * kStageScales);
#pragma unroll
  for (int i = 0; i < 4; ++i) load_codes(t.h, t.h_at, half, smem + buf * kHalfBytes, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) load_codes(t.w, t.w_at, half, smem + buf * kHalfBytes + kHalfPanel, i);
}

// Loads that a wave has in flight behind those that a half stage waits for: two
// half stages, one of them with its stage's scales, and, where the last tile's
// 32 stores were issued since, those.
constexpr int kInFlight = 2 * 8 + 1;
constexpr int kStores = 2 * kMB * kNB;
static_assert(kInFlight + kStores <= 63, "the counter holds 6 bits");

// Waits until all but the newest n of this wave's loads and stores are done
// (they complete in order) and its LDS reads are, then for the workgroup.
template <int n>
__device__ __forceinline__ void half_barrier() {
  static_assert(n == 0 || n == kInFlight || n == kInFlight + kStores, "one of the three counts");
  if constexpr (n == 0)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (n == kInFlight)
    asm volatile("s_waitcnt vmcnt(17) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    asm volatile("s_waitcnt vmcnt(49) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Fragment of step kk (0, 1) of a half stage of a wave's tile i (32 rows, 64 deep).
__device__ __forceinline__ Frag frag(const uint8_t* __restrict__ panel, int first, int i, int kk) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const Frag*>(panel + ((first + i) * kHalfSteps + kk) * kStepBytes + lane * 16);
}

__device__ __forceinline__ int scale_word(const uint8_t* __restrict__ scales, int first, int i) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const int*>(scales + (first + i) * kScaleBytes + lane * 4);
}

struct Scales {
  int h[kMB];
  int w[kNB];
};

struct Ahead {      // of the half stage to come: its fragments, and its stage's scales
  Frag a[kHalfSteps][kMB];
  Frag b[kHalfSteps][kNB];
  Scales sc;
};

// One step: 16 instructions, each followed by its share of the reads for the
// same step of the next half stage (8 fragments; with kk 1 and 2 of a stage's
// second half also the next stage's 8 words of scales) and of the loads of the
// half stage four ahead (8, and a stage's scales).
// kFirst: the tile's first step, whose accumulators are the instruction's
// constant 0 (256 registers need no clearing).
template <int kk, bool kFirst>
__device__ __forceinline__ void mma_step(const Frag (&a)[kMB], const Frag (&b)[kNB], const Scales& sc,
                                         f32x16 (&acc)[kMB][kNB], const uint8_t* __restrict__ from,
                                         const uint8_t* __restrict__ scales, int fm, int fn, Frag (&na)[kMB],
                                         Frag (&nb)[kNB], Scales& next, const Tile& t, int half, int buf,
                                         uint8_t* __restrict__ smem) {
  constexpr int step = kk % kHalfSteps;
#pragma unroll
  for (int s = 0; s < kMB * kNB; ++s) {
    const int i = s / kNB, j = s % kNB;
    if constexpr (kFirst) {
      const f32x16 zero = {};
      acc[i][j] = mma<kk>(b[j], a[i], zero, sc.w[j], sc.h[i]);
    } else {
      acc[i][j] = mma<kk>(b[j], a[i], acc[i][j], sc.w[j], sc.h[i]);
    }
    if (s < kMB)
      na[s] = frag(from, fm, s, step);
    else if (s < kMB + kNB)
      nb[s - kMB] = frag(from + kHalfPanel, fn, s - kMB, step);
    else if (kk == 2 && s < kMB + kNB + kMB)
      next.h[s - kMB - kNB] = scale_word(scales, fm, s - kMB - kNB);
    else if (kk == 2)
      next.w[s - 2 * kMB - kNB] = scale_word(scales + kPanelScales, fn, s - 2 * kMB - kNB);
    if (kk == 0 && s == 1)
      load_scales(t, half < 0 ? -1 : half >> 1, smem + kOffScales + (buf >> 1) * kStageScales);
    if ((s & 3) == 2) {
      if (step == 0)
        load_codes(t.h, t.h_at, half, smem + buf * kHalfBytes, s >> 2);
      else
        load_codes(t.w, t.w_at, half, smem + buf * kHalfBytes + kHalfPanel, s >> 2);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The fragments of a landed half stage and its stage's scales.
__device__ __forceinline__ void read_first(const uint8_t* __restrict__ smem, int buf, int fm, int fn, Ahead& f) {
  const uint8_t* panel = smem + buf * kHalfBytes;
  const uint8_t* scales = smem + kOffScales + (buf >> 1) * kStageScales;
#pragma unroll
  for (int kk = 0; kk < kHalfSteps; ++kk) {
#pragma unroll
    for (int i = 0; i < kMB; ++i) f.a[kk][i] = frag(panel, fm, i, kk);
#pragma unroll
    for (int j = 0; j < kNB; ++j) f.b[kk][j] = frag(panel + kHalfPanel, fn, j, kk);
  }
#pragma unroll
  for (int i = 0; i < kMB; ++i) f.sc.h[i] = scale_word(scales, fm, i);
#pragma unroll
  for (int j = 0; j < kNB; ++j) f.sc.w[j] = scale_word(scales + kPanelScales, fn, j);
}

// The tile's K loop takes 46-48,000 cycles at d = 4096 (the instructions alone
// 32,768), its store 6-7,000, the step to the next tile 2,000, at 1.75-1.85 GHz:
// the chip's power sets the clock. Without the loads into LDS the loop would take
// 39,300, and 42,700 with every load from one place; waiting for them costs
// nothing (counted waits against none), nor do the fragment reads.
//
// Products of one tile. Half stage x of the tile lives in LDS buffer (2 par +
// x) % 4. While it is multiplied, the fragments of half stage x + 1 are read;
// the barrier before it waits for x + 1 to land in LDS and for every wave's
// reads of x's buffer (made one half stage before), so that buffer takes half
// stage x + 4: three half stages, about 3000 cycles, cover a load. Behind the
// tile's end x + 1 and x + 4 are the next tile's (tn), whose half stages 0 to 3
// are in flight or landed on return and whose first fragments are read.
// stored: the wave's last 32 stores may still be in flight.
template <bool kFirst>
__device__ __forceinline__ void stage_products(const Tile& t, const Tile& tn, bool ahead, int n, int kt, int par,
                                               bool stored, uint8_t* __restrict__ smem, int fm, int fn,
                                               f32x16 (&acc)[kMB][kNB], Ahead& f) {
  const int buf = 2 * ((kt + par) & 1);       // of this stage's first half; the next stage's are the other two
  const bool mine = kt + 2 < n;
  const Tile q = mine ? t : tn;
  const int k2 = mine ? 2 * (kt + 2) : (ahead ? 2 * (kt + 2 - n) : -2);
  Ahead o;
  const uint8_t* second = smem + (buf + 1) * kHalfBytes;
  if (stored && kt < 2)
    half_barrier<kInFlight + kStores>();
  else
    half_barrier<kInFlight>();
  mma_step<0, kFirst>(f.a[0], f.b[0], f.sc, acc, second, nullptr, fm, fn, o.a[0], o.b[0], o.sc, q, k2, buf, smem);
  mma_step<1, false>(f.a[1], f.b[1], f.sc, acc, second, nullptr, fm, fn, o.a[1], o.b[1], o.sc, q, k2, buf, smem);
  const uint8_t* third = smem + (buf ^ 2) * kHalfBytes;
  const uint8_t* scales = smem + kOffScales + ((buf ^ 2) >> 1) * kStageScales;
  if (kFirst && stored)
    half_barrier<kInFlight + kStores>();
  else
    half_barrier<kInFlight>();
  mma_step<2, false>(o.a[0], o.b[0], f.sc, acc, third, scales, fm, fn, f.a[0], f.b[0], o.sc, q, k2 + 1, buf + 1, smem);
  mma_step<3, false>(o.a[1], o.b[1], f.sc, acc, third, scales, fm, fn, f.a[1], f.b[1], o.sc, q, k2 + 1, buf + 1, smem);
  f.sc = o.sc;
}

__device__ __forceinline__ void tile_products(const TileGeo& g, const Tile& t, const Tile& tn, bool next, int par,
                                              bool stored, uint8_t* __restrict__ smem, int fm, int fn,
                                              f32x16 (&acc)[kMB][kNB], Ahead& f) {
  const int n = g.g.steps4;
  const bool ahead = next && n >= 2;
  stage_products<true>(t, tn, ahead, n, 0, par, stored, smem, fm, fn, acc, f);
  for (int kt = 1; kt < n; ++kt) stage_products<false>(t, tn, ahead, n, kt, par, stored, smem, fm, fn, acc, f);
}

// `mine` in the lanes of `keep`, else the `other` of lane l ^ (1 << b): one
// select with its operand taken across the quad (written out, because the
// compiler leaves the exchange and the select apart, twice the instructions;
// the nop covers the distance that an exchange needs from its operand's write).
template <int b>
__device__ __forceinline__ u32x4 keep_or_take(const u32x4& mine, const u32x4& other, uint64_t keep) {
  uint32_t x, y, z, w;
  if constexpr (b == 0)
    asm("s_mov_b64 vcc, %[keep]\n\ts_nop 1\n\t"
        "v_cndmask_b32_dpp %[x], %[ox], %[mx], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[y], %[oy], %[my], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[z], %[oz], %[mz], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[w], %[ow], %[mw], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf"
        : [x] "=&v"(x), [y] "=&v"(y), [z] "=&v"(z), [w] "=&v"(w)
        : [keep] "s"(keep), [mx] "v"(mine.x), [my] "v"(mine.y), [mz] "v"(mine.z), [mw] "v"(mine.w), [ox] "v"(other.x),
          [oy] "v"(other.y), [oz] "v"(other.z), [ow] "v"(other.w)
        : "vcc");
  else
    asm("s_mov_b64 vcc, %[keep]\n\ts_nop 1\n\t"
        "v_cndmask_b32_dpp %[x], %[ox], %[mx], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[y], %[oy], %[my], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[z], %[oz], %[mz], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %[w], %[ow], %[mw], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf"
        : [x] "=&v"(x), [y] "=&v"(y), [z] "=&v"(z), [w] "=&v"(w)
        : [keep] "s"(keep), [mx] "v"(mine.x), [my] "v"(mine.y), [mz] "v"(mine.z), [mw] "v"(mine.w), [ox] "v"(other.x),
          [oy] "v"(other.y), [oz] "v"(other.z), [ow] "v"(other.w)
        : "vcc");
  return u32x4{x, y, z, w};
}

// Stores a wave's 128 x 128 logits; pads -inf. A part inside the matrix takes
// kStores stores in every lane and returns true (uniform across the wave); at
// an edge all stores are done on return. Inside, lanes of a quad exchange
// 16-byte pieces first (bit 0 of the lane for the piece, bit 1 for the block of
// 32 columns), so that 8 lanes write a row's 128 bytes with one instruction: as
// the accumulators lie, every lane of a store writes another row, which took
// 11,300 cycles a tile.
__device__ __forceinline__ bool tile_store(const Geo& g, int64_t row0, int64_t col0, const f32x16 (&acc)[kMB][kNB],
                                           uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int h = lane >> 5;
  if (row0 + kMB * 32 <= g.n_rows && col0 + kNB * 32 <= g.vocab_real) {
    constexpr uint64_t kClear0 = 0x5555555555555555ull, kClear1 = 0x3333333333333333ull;  // lanes with the bit clear
    const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0;
    uint16_t* base = out + (row0 + (lane & 28)) * g.ldo + col0 + 32 * (b1 ? 1 : 0) + 16 * h + 8 * (b0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
#pragma unroll
      for (int j = 0; j < kNB; j += 2) {
        u32x4 even[2], odd[2];  // rows of even and of odd number, of block j + k: piece b0
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[8];
          rlk::block_words(acc[i][j + k], w);
          const u32x4 p0 = {w[0], w[1], w[2], w[3]}, p1 = {w[4], w[5], w[6], w[7]};
          even[k] = keep_or_take<0>(p0, p1, kClear0);
          odd[k] = keep_or_take<0>(p1, p0, ~kClear0);
        }
        uint16_t* dst = base + static_cast<int64_t>(i * 32) * g.ldo + j * 32;
        *reinterpret_cast<u32x4*>(dst) = keep_or_take<1>(even[0], even[1], kClear1);
        *reinterpret_cast<u32x4*>(dst + g.ldo) = keep_or_take<1>(odd[0], odd[1], kClear1);
        *reinterpret_cast<u32x4*>(dst + 2 * g.ldo) = keep_or_take<1>(even[1], even[0], ~kClear1);
        *reinterpret_cast<u32x4*>(dst + 3 * g.ldo) = keep_or_take<1>(odd[1], odd[0], ~kClear1);
      }
    }
    return true;
  }
#pragma unroll
  for (int i = 0; i < kMB; ++i) {
    const int64_t row = row0 + i * 32 + (lane & 31);
    uint16_t* dst = out + row * g.ldo;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      uint32_t w[8];
      rlk::block_words(acc[i][j], w);
      const int64_t c = col0 + j * 32 + 16 * h;
      if (row < g.n_rows && c < g.vocab_padded) {
        rlk::store8(g.vocab_real, dst + c, c, w[0], w[1], w[2], w[3]);
        rlk::store8(g.vocab_real, dst + c + 8, c + 8, w[4], w[5], w[6], w[7]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  return false;
}

__global__ __launch_bounds__(kTilesThreads) void k_mx4_tiles(TileGeo g, uint16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmemBytes];
  const int n = g.g.steps4;
  Walk at(g);
  if (!at.find(g)) return;  // uniform across the workgroup
  const int wave = wave_id();
  const int fm = (wave & 1) * kMB;
  const int fn = (wave >> 1) * kNB;
  Tile t = make_tile(g, at);
  int par = 0;
  bool stored = false;
  Ahead f;
#pragma unroll
  for (int x = 0; x < 4; ++x) load_half(t, n > 1 || x < 2 ? x : -2, x, smem);
  half_barrier<0>();
  read_first(smem, 0, fm, fn, f);
  int m_t = at.m_t, n_t = at.n_t;
  at.step();
  bool more = at.find(g);
  Tile tn = more ? make_tile(g, at) : t;
  while (true) {
    f32x16 acc[kMB][kNB];
    tile_products(g, t, tn, more, par, stored, smem, fm, fn, acc, f);
    stored = tile_store(g.g, static_cast<int64_t>(m_t) * BM + fm * 32, static_cast<int64_t>(n_t) * BN + fn * 32, acc, out);
    if (!more) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is in flight when the workgroup ends
      break;
    }
    par = (par + n) & 1;
    m_t = at.m_t;
    n_t = at.n_t;
    t = tn;
    at.step();
    more = at.find(g);
    tn = more ? make_tile(g, at) : t;
    if (n == 1) {
      // a tile of one stage could not load the next one in its loop: the other
      // stage's buffers, which every wave has left (they were read behind the
      // last barrier, as fragments that are replaced here)
      half_barrier<0>();
#pragma unroll
      for (int x = 0; x < 2; ++x) load_half(t, x, 2 * par + x, smem);
      half_barrier<0>();
      stored = false;
      read_first(smem, 2 * par, fm, fn, f);
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

template <int NB>
static void launch_stream_blocks(const Geo& g, const uint16_t* hidden, int64_t ldh, int d, uint16_t* out, hipStream_t stream) {
  const int tiles = static_cast<int>(g.vocab_padded / kTileRows);  // at most 2^25
  const int w_tiles = static_cast<int>(row_tiles(g.vocab_real));
  constexpr int kMost = stream_most(NB);
  const auto run = [&](auto kernel, int split) {
    const int teams = stream_waves(NB) / split;
    const int wanted = (tiles + teams - 1) / teams, most = 256 * stream_groups(NB);
    kernel<<<dim3(static_cast<unsigned>(wanted < most ? wanted : most)), dim3(stream_waves(NB) * 64), 0, stream>>>(
        g, hidden, ldh, d, tiles, w_tiles, out);
  };
  // as few parts of d as the registers hold
  if (g.steps4 <= 1)
    run(k_mx4_stream<NB, 1, 1>, 1);
  else if (g.steps4 <= 2)
    run(k_mx4_stream<NB, 2, 1>, 1);
  else if (g.steps4 <= kMost)
    run(k_mx4_stream<NB, kMost, 1>, 1);
  else if (g.steps4 <= 2 * kMost)
    run(k_mx4_stream<NB, kMost, 2>, 2);
  else if (g.steps4 <= 4 * kMost)
    run(k_mx4_stream<NB, kMost, 4>, 4);
  else if constexpr (8 * kMost <= kStreamSteps4)
    run(k_mx4_stream<NB, kMost, 8>, 8);
}

static void launch_stream(const Geo& g, int blocks, const uint16_t* hidden, int64_t ldh, int d, uint16_t* out,
                          hipStream_t stream) {
  if (blocks == 1)
    launch_stream_blocks<1>(g, hidden, ldh, d, out, stream);
  else if (blocks == 2)
    launch_stream_blocks<2>(g, hidden, ldh, d, out, stream);
  else
    launch_stream_blocks<4>(g, hidden, ldh, d, out, stream);
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
  const int blocks_of_rows = static_cast<int>(row_tiles(n_rows) < 8 ? row_tiles(n_rows) : 8);
  const bool streamed = blocks_of_rows <= kStreamBlocks && g.steps4 <= kStreamSteps4;
  if (!(streamed && blocks_of_rows == 1) &&
      (st = launch_quantize(hidden, n_rows, d_model, hidden_stride, hc, hs, nullptr, 0, stream)) != RLK_OK)
    return st;
  if (streamed) {
    launch_stream(g, blocks_of_rows, hidden, hidden_stride, static_cast<int>(d_model), logits_out, stream);
    return launched();
  }
  if (n_rows > kRowsMost || (blocks_of_rows > 1 && layout->vocab_padded >= kRowsTiles * BN)) {
    TileGeo t;
    t.g = g;
    t.m_tiles = static_cast<int>((n_rows + BM - 1) / BM);                       // at most 2^14
    t.n_tiles = static_cast<int>((layout->vocab_padded + BN - 1) / BN);         // at most 2^22
    const int bands = (t.m_tiles + 3) / 4;
    t.band = (t.m_tiles + bands - 1) / bands;                                   // as even as they go
    t.chunk = bands > 1 ? 8 : t.n_tiles;
    t.h_end = row_tiles(n_rows);
    t.w_end = row_tiles(layout->vocab_real);
    // one workgroup for each of 256 compute units (its LDS fills one), each walking over its tiles
    k_mx4_tiles<<<dim3(kXcds * kGroup), dim3(kTilesThreads), 0, stream>>>(t, logits_out);
    return launched();
  }
  const int64_t col_tiles = layout->vocab_padded / kRowsCols;
  const int64_t n_work = col_tiles * row_tiles(n_rows);
  const int64_t blocks = (n_work + kRowsThreads / 64 - 1) / (kRowsThreads / 64);  // at most 2^22 (beyond 32 rows: fewer than 512 column tiles)
  k_mx4_rows<<<dim3(static_cast<unsigned>(blocks)), dim3(kRowsThreads), 0, stream>>>(g, col_tiles, n_work, logits_out);
  return launched();
}

}  // extern "C"
