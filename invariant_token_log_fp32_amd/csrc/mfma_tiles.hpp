// 256 x 256 tiles of a BF16 product on the matrix cores, operands in either
// memory order: a workgroup of 4 waves (one per SIMD), each 128 x 128 as 4 x 4
// blocks of v_mfma_f32_32x32x16_bf16, K in 64-wide stages through
// double-buffered LDS, panels loaded from global memory straight into LDS.
//
//   out[m][n] = sum_k A[m][k] * B[n][k],  A = a[m * lda + k] (K contiguous) or
//   a[k * lda + m] (K across rows); the same for B.
//
// Operand with K contiguous: an LDS stage is 256 rows of 64 values (128
// bytes), the 16-byte chunks of row r permuted by an XOR with swz(r); one
// ds_read_b128 gives a lane its 8 values of a K step.
//
// Operand with K across rows: a stage is 64 rows (k) of 256 values (512
// bytes), read with ds_read_b64_tr_b16: 16 lanes take a 4 (k) x 16 block, and
// lane t receives column t's 4 values; two of them are a K step's 8. The four
// rows of a block lie 512 bytes apart, in the same banks, so the 32-byte
// pieces of row k are permuted by an XOR with 2 (k % 4): the 32 lanes that
// read together then cover all 64 banks once.
//
// Order of a sum: increasing k, 16 a matrix instruction, the accumulator
// carried, the second operand's fragment (B) first: bit for bit that of
// rlk_linear for the same values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16_store.hpp"
#include "logp_device.hpp"

namespace rlk_tiles {

using rlk::f32x16;

constexpr int BM = 256;
constexpr int BN = 256;
constexpr int BK = 64;                  // K per LDS stage
constexpr int kThreads = 256;           // 4 waves, 2 x 2
constexpr int kWaveM = 128;
constexpr int kWaveN = 128;
constexpr int kMB = kWaveM / 32;        // 32 x 32 blocks per wave
constexpr int kNB = kWaveN / 32;
constexpr int kSteps = BK / 16;         // K steps per stage
constexpr int kStage = BM * BK;         // values per operand and stage
constexpr int kSmem = 4 * kStage;       // two stages of both operands: 128 KB
constexpr int kXcds = 8;
// Tiles of an XCD's 32 compute units: 4 x 8, so that its L2 serves each panel
// to several of them (as in rlk_linear).
constexpr int kGM = 4;
constexpr int kGN = 8;

static_assert(BM == BN && kSteps == 4 && kMB == 4 && kNB == 4, "the step below is written out for this shape");

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef f32x16 Acc[kMB][kNB];
typedef __attribute__((address_space(3))) void* LdsPtr;

constexpr int kRsrcWord3 = 0x00020000;  // gfx9 raw buffer: 32-bit data format, no swizzle

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6); }

__host__ __device__ __forceinline__ constexpr int swz(int r) { return (((r >> 1) & 3) << 1) | ((r >> 3) & 1); }

// One operand of one tile: where its first stage begins and what may be read.
struct Panel {
  const uint16_t* p;
  int lim;  // K contiguous: bytes from p to the end of the last row's K; K across rows: bytes of a row from p on
};

// K contiguous: `rows` valid rows from p on, k values each.
__device__ __forceinline__ Panel panel_rows(const uint16_t* p, int rows, int ld, int k) {
  return Panel{p, (rows > 0 && k > 0) ? ((rows - 1) * ld + k) * 2 : 0};
}

// K across rows: `cols` valid columns from p on (at least one).
__device__ __forceinline__ Panel panel_cols(const uint16_t* p, int64_t cols) {
  return Panel{p, static_cast<int>(cols < BN ? cols : BN) * 2};
}

// Stage st of a panel as a buffer resource whose range check returns zeros for
// rows past the operand's end, and for k past `k_end` where K runs across rows;
// with `any` false one that loads nothing.
template <bool kAcross>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t stage_of(const Panel& q, int ld, int k_end, int st, bool any) {
  const int64_t skip = kAcross ? static_cast<int64_t>(st) * BK * ld : st * BK;
  int rec;
  if (kAcross) {
    const int left = k_end - st * BK;
    const int rows = left < BK ? left : BK;
    rec = rows > 0 ? (rows - 1) * ld * 2 + q.lim : 0;
  } else {
    rec = q.lim - st * BK * 2;
  }
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(q.p + skip), 0, any && rec > 0 ? rec : 0, kRsrcWord3);
}

// This lane's byte offsets into a stage for the 8 loads that fill it: loads 0
// and 1, and the distance between loads i and i + 2. Load i of wave w fills
// 1 KB of LDS in lane order, from 1 KB * (8 w + i) on.
struct Offsets {
  int at[2];
  int step;
};

template <bool kAcross>
__device__ __forceinline__ Offsets offsets_for(int ld) {
  const int l = static_cast<int>(threadIdx.x) & 63;
  const int w = static_cast<int>(threadIdx.x) >> 6;
  Offsets o;
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    if (kAcross) {  // rows k = 16 w + 2 i and the next, 32 chunks each
      const int k = 16 * w + 2 * par + (l >> 5);
      const int c = (l & 31) ^ (4 * (k & 3));
      o.at[par] = k * ld * 2 + c * 16;
    } else {        // rows 64 w + 8 i .. + 7, 8 chunks each
      const int r = 64 * w + 8 * par + (l >> 3);
      const int c = (l & 7) ^ swz(r);
      o.at[par] = r * ld * 2 + c * 16;
    }
  }
  o.step = (kAcross ? 4 : 16) * ld * 2;
  // without this the offsets of all loads are kept apart, and spilled
  asm volatile("" : "+v"(o.at[0]), "+v"(o.at[1]));
  return o;
}

__device__ __forceinline__ void load_one(__amdgpu_buffer_rsrc_t r, const Offsets& o, uint16_t* __restrict__ s, int i) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)(s + (8 * wave_id() + i) * 512), 16,
                                           o.at[i & 1] + (i >> 1) * o.step, 0, 0, 0);
}

__device__ __forceinline__ void load_stage(__amdgpu_buffer_rsrc_t r, const Offsets& o, uint16_t* __restrict__ s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) load_one(r, o, s, i);
}

// Waits for this wave's LDS operations and panel loads, then for the workgroup.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// LDS addresses of a wave's fragments in one operand's current stage: lane l
// takes row or column 32 i + l % 32 of block i, k = 16 kk + 8 (l / 32) .. + 7 in K
// step kk. The chunk permutations make four of them: one a K step where K is
// contiguous (blocks lie 4 KB apart), one a block where it runs across rows (K
// steps lie 8 KB apart).
struct FragAt {
  uint32_t at[4];
};

constexpr uint32_t kStageBytes = kStage * 2;

template <bool kAcross>
__device__ __forceinline__ FragAt frag_at(const uint16_t* stage, int w) {
  const int lane = threadIdx.x & 63;
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LdsPtr)(const_cast<uint16_t*>(stage))));
  FragAt f;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if (kAcross) {
      const int q = (lane >> 2) & 3;  // row of the 4 x 16 block that this lane's address names
      f.at[n] = base + ((8 * (lane >> 5) + q) * BN + (w * 8 + ((lane >> 4) & 1) + (n ^ q) * 2) * 16 + (lane & 3) * 4) * 2;
    } else {
      const int fr = lane & 31;
      f.at[n] = base + ((w * kWaveM + fr) * BK + ((2 * n + (lane >> 5)) ^ swz(fr)) * 8) * 2;
    }
    asm volatile("" : "+v"(f.at[n]));  // kept in registers, not formed again for every read
  }
  return f;
}

typedef __attribute__((address_space(3))) s16x4* LdsTr;
typedef __attribute__((address_space(3))) const bf16x8* LdsFrag;

template <bool kAcross>
__device__ __forceinline__ bf16x8 read_frag(const FragAt& f, int i, int kk) {
  if (kAcross) {
    const uint32_t p = f.at[i] + kk * 16 * BN * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(p + 4 * BN * 2));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return *(LdsFrag)(f.at[kk] + i * 32 * BK * 2);
}

template <bool kTA, bool kTB>
__device__ __forceinline__ void load_frags(const FragAt& pa, const FragAt& pb, int kk, bf16x8 (&a)[kMB],
                                           bf16x8 (&b)[kNB]) {
#pragma unroll
  for (int i = 0; i < kMB; ++i) a[i] = read_frag<kTA>(pa, i, kk);
#pragma unroll
  for (int j = 0; j < kNB; ++j) b[j] = read_frag<kTB>(pb, j, kk);
}

// One K step: 16 matrix instructions, with the fragments of the step after
// next read between them, and, in steps that carry panel loads, one of the 8
// loads of a panel after every other instruction.
template <bool kLoads, bool kTA, bool kTB>
__device__ __forceinline__ void mma_step(const bf16x8 (&a)[kMB], const bf16x8 (&b)[kNB], Acc& acc, const FragAt& pa,
                                         const FragAt& pb, int kk, bf16x8 (&na)[kMB], bf16x8 (&nb)[kNB],
                                         __amdgpu_buffer_rsrc_t rs, const Offsets& o, uint16_t* __restrict__ ld_to) {
#pragma unroll
  for (int t = 0; t < kMB * kNB; ++t) {
    const int i = t / kNB;
    const int j = t % kNB;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    if (t < kMB)
      na[t] = read_frag<kTA>(pa, t, kk);
    else if (t < kMB + kNB)
      nb[t - kMB] = read_frag<kTB>(pb, t - kMB, kk);
    if (kLoads && (t & 1) == 0) load_one(rs, o, ld_to, t >> 1);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A tile's product: panels, the operands' strides and the end of K.
struct TileIn {
  Panel a, b;
  int k_end;
};

__device__ __forceinline__ int stages_of(int k_end) {
  const int n = (k_end + BK - 1) / BK;
  return n > 0 ? n : 1;  // an empty sum still goes through one stage, of zeros
}

// Stages 0 and 1 of a tile into LDS buffers par and par ^ 1.
template <bool kTA, bool kTB>
__device__ __forceinline__ void prefetch_tile(const TileIn& t, int lda, int ldb, const Offsets& oa, const Offsets& ob,
                                              int par, uint16_t* __restrict__ smem) {
  const bool two = stages_of(t.k_end) > 1;
  load_stage(stage_of<kTA>(t.a, lda, t.k_end, 0, true), oa, smem + par * kStage);
  load_stage(stage_of<kTB>(t.b, ldb, t.k_end, 0, true), ob, smem + (2 + par) * kStage);
  load_stage(stage_of<kTA>(t.a, lda, t.k_end, 1, two), oa, smem + (par ^ 1) * kStage);
  load_stage(stage_of<kTB>(t.b, ldb, t.k_end, 1, two), ob, smem + (2 + (par ^ 1)) * kStage);
}

// The sums of one tile into acc. Stage kt lives in LDS buffer (kt + par) & 1,
// which pa, pb point into on entry; stages 0 and 1 are loaded or in flight then
// and the fragments of steps 0 and 1 in fa[0..1], fb[0..1]. Fragments are read
// two steps ahead, so a stage's buffer is free after step 1: one barrier there,
// after the next stage's loads have landed; steps 2 and 3 then load the stage
// after next (in the last two stages: stages 0 and 1 of the next tile, when there
// is one) into the freed buffer. Block (i, j): element 4 q + e of lane l is row
// 32 i + l % 32, column 32 j + 8 q + 4 (l / 32) + e of the wave's part.
template <bool kTA, bool kTB>
__device__ __forceinline__ void tile_sums(const TileIn& t, const TileIn& tn, bool next, int lda, int ldb,
                                          const Offsets& oa, const Offsets& ob, int par, FragAt& pa, FragAt& pb,
                                          uint16_t* __restrict__ smem, Acc& acc, bf16x8 (&fa)[kSteps][kMB],
                                          bf16x8 (&fb)[kSteps][kNB]) {
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int kt_n = stages_of(t.k_end);
  const bool ahead = next && kt_n >= 2;
  for (int kt = 0; kt < kt_n; ++kt) {
    const int cur = (kt + par) & 1;
    uint16_t* ca = smem + cur * kStage;
    const bool own = kt + 2 < kt_n;
    const int st = own ? kt + 2 : kt + 2 - kt_n;
    const Panel qa = {own ? t.a.p : tn.a.p, own ? t.a.lim : tn.a.lim};
    const Panel qb = {own ? t.b.p : tn.b.p, own ? t.b.lim : tn.b.lim};
    const int k_end = own ? t.k_end : tn.k_end;
    const __amdgpu_buffer_rsrc_t ra = stage_of<kTA>(qa, lda, k_end, st, own || ahead);
    const __amdgpu_buffer_rsrc_t rb = stage_of<kTB>(qb, ldb, k_end, st, own || ahead);
    mma_step<false, kTA, kTB>(fa[0], fb[0], acc, pa, pb, 2, fa[2], fb[2], ra, oa, ca);
    mma_step<false, kTA, kTB>(fa[1], fb[1], acc, pa, pb, 3, fa[3], fb[3], ra, oa, ca);
    stage_barrier();
    const uint32_t turn = cur ? 0u - kStageBytes : kStageBytes;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      pa.at[n] += turn;
      pb.at[n] += turn;
    }
    mma_step<true, kTA, kTB>(fa[2], fb[2], acc, pa, pb, 0, fa[0], fb[0], ra, oa, ca);
    mma_step<true, kTA, kTB>(fa[3], fb[3], acc, pa, pb, 1, fa[1], fb[1], rb, ob, ca + 2 * kStage);
  }
}

// Tile u of m_tiles x n_tiles, every index a tile: bands of kGN tiles along n,
// in a band groups of kGM x kGN, in a group m first.
__device__ __forceinline__ void tile_at(int u, int m_tiles, int n_tiles, int& m, int& n) {
  const int band = u / (kGN * m_tiles);
  const int left = n_tiles - band * kGN;
  const int bn = left < kGN ? left : kGN;
  const int r = u - band * kGN * m_tiles;
  const int g = r / (kGM * bn);
  const int mleft = m_tiles - g * kGM;
  const int bm = mleft < kGM ? mleft : kGM;
  const int l = r - g * kGM * bn;
  m = g * kGM + l % bm;
  n = band * kGN + l / bm;
}

// First tile index of workgroup b, which runs on XCD b % 8: the XCD's
// workgroups take neighbouring tiles (grid: a multiple of 8).
__device__ __forceinline__ int first_tile() {
  const int b = static_cast<int>(blockIdx.x);
  return (b % kXcds) * (static_cast<int>(gridDim.x) / kXcds) + b / kXcds;
}

}  // namespace rlk_tiles
