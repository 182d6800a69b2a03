// Gradient of the fused linear + token logprob on gfx950, and the C ABI
// declared in include/rlk_linear_grad.h.
//
// Passages: RL-Kernel page "H100 canonical CP backward validation", Change
// section (the training step back-propagates through the logprobs), and page
// "Reproduce and profile the Qwen3-8B TP4/CP2 experiment" (the linear-logp
// backend; summaries per canonical vocabulary shard in fixed order).
//
// With G the gradient of the BF16 logits x = bf16(h w^T):
//   grad_hidden = G w,  grad_weight = G^T h
// three products of the same size, none of which keeps more of x or G than a
// few canonical vocabulary shards (an eighth of the vocabulary each).
//
// Kernels, in order:
//   k_rows     per row the coefficients of G (those of rlk_logp_backward); rows
//              without a gradient are left out, the others numbered in order
//              (one workgroup: a running count over 1024 rows at a time; 4 us up to
//              640 rows, 23 for 8192)
//   k_gather   the hidden states of the rows that remain, side by side; zeros
//              into grad_hidden of the others
//   k_product  <kLogits> x of some shards (bit for bit rlk_linear's), turned
//              into G in the accumulators and stored in BF16
//              <kHidden> G times the projection's rows, a partial sum for each
//              shard
//   k_weight   G^T times the hidden states
//   k_combine  a row's partial sums added in the fixed order
// The products run on the tiles of mfma_tiles.hpp, one workgroup a compute unit
// looping over its tiles. What bounds them, at 4096 columns of hidden states and a
// vocabulary of 151936: one row reads the projection twice and writes its gradient in
// 0.78 ms (4.8 TB/s; a bare read and a fill reach 6.9, which would be 0.54): the logits pass takes
// 256 to 316 us where grad_hidden takes 211 for the same bytes, of which a slice of the
// logits has 64 in a row and one of grad_hidden 256. 8192 rows take 22.7 ms (1.35 PFLOP/s)
// or, on a warm GPU, 24.6, as long as the three library products alone in the same loop
// (1.24): the power limit; in between, rounds of tiles that the compute units share
// unevenly (640 rows, grad_hidden alone, 1.50 ms: 1.06 PFLOP/s). Both operands of kWeight and the projection in kHidden
// run across K in memory; they are transposed on the way from LDS to registers,
// so no transposed copy is written.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "bf16_store.hpp"
#include "logp_device.hpp"
#include "mfma_tiles.hpp"
#include "rlk_linear_grad.h"
#include "rlk_logp.h"

namespace rlk_lin_grad {

using rlk::u32x4;
using namespace rlk_tiles;

constexpr int kShards = rlk::kShards;
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxLd = int64_t(1) << 21;
constexpr int64_t kMaxVocab = int64_t(1) << 22;  // 256 rows of a shard's G: byte offsets fit 31 bits
constexpr int kMaxD = 65536;

// What turns x of one row into G: G_j = s_r 2^(x_j c + a_r) + [x_j >= thr] s_p 2^(x_j c + a_p),
// g_t in the target column.
struct alignas(16) RowCoef {
  float c, a_r, s_r, a_p;
  float s_p, thr, g_t;
  int32_t target;  // global column, -1: none
};

// The row's coefficients; false when the row has no gradient.
__device__ __forceinline__ bool row_coef(int64_t row, int64_t vocab_real, const float* __restrict__ temperature,
                                         const int64_t* __restrict__ target, const float* __restrict__ ref_logp,
                                         const float* __restrict__ lse, const float* __restrict__ grad_ref,
                                         const float* __restrict__ policy_logp,
                                         const rlk_support_state* __restrict__ support,
                                         const float* __restrict__ grad_policy, RowCoef& R) {
  const float gr = grad_ref ? grad_ref[row] : 0.0f;
  const float gp = grad_policy ? grad_policy[row] : 0.0f;
  if (gr == 0.0f && gp == 0.0f) return false;
  const float t = temperature[row];
  const int64_t tg = target[row];
  const float ref = grad_ref ? ref_logp[row] : 0.0f;
  const int status = grad_policy ? support[row].status : 1;
  const bool invalid = !rlk::temperature_valid(t) || tg < 0 || tg >= vocab_real || ref != ref || status == -2;
  if (!invalid && t == 0.0f) return false;
  R = RowCoef{0.0f, 0.0f, NAN, 0.0f, 0.0f, INFINITY, NAN, -1};  // NaN in every real column
  if (invalid || (gp != 0.0f && status == -1)) return true;
  R.c = rlk::kLog2e / t;
  // without a reference term its power is 0 (a finite one could overflow beside s_r = 0)
  R.a_r = gr != 0.0f ? static_cast<float>(-static_cast<double>(lse[row]) * 1.4426950408889634) : -INFINITY;
  R.s_r = -gr / t;
  const float gpe = status == 1 ? gp : 0.0f;
  R.s_p = -gpe / t;
  float tpol = 0.0f;
  if (gpe != 0.0f) {
    const rlk_support_state st = support[row];
    R.a_p = static_cast<float>(-static_cast<double>(st.lse_support) * 1.4426950408889634);
    R.thr = st.threshold;
    tpol = gpe * -expm1f(policy_logp[row]);
  }
  const float tref = gr != 0.0f ? gr * -expm1f(ref) : 0.0f;
  R.g_t = (tref + tpol) / t;
  R.target = static_cast<int32_t>(tg);
  return true;
}

constexpr int kRowThreads = 1024;

// coef[p], row_of[p] for the p-th row with a gradient; place[row] = p or -1; *n_act.
__global__ __launch_bounds__(kRowThreads) void k_rows(int64_t n_rows, int64_t vocab_real,
                                                      const float* __restrict__ temperature,
                                                      const int64_t* __restrict__ target,
                                                      const float* __restrict__ ref_logp,
                                                      const float* __restrict__ lse,
                                                      const float* __restrict__ grad_ref,
                                                      const float* __restrict__ policy_logp,
                                                      const rlk_support_state* __restrict__ support,
                                                      const float* __restrict__ grad_policy,
                                                      RowCoef* __restrict__ coef, int32_t* __restrict__ row_of,
                                                      int32_t* __restrict__ place, int32_t* __restrict__ n_act) {
  __shared__ int count[2][kRowThreads / 64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  int before = 0;
  int buf = 0;
  for (int64_t at = 0; at < n_rows; at += kRowThreads, buf ^= 1) {  // uniform
    const int64_t row = at + threadIdx.x;
    RowCoef R;
    const bool live = row < n_rows && row_coef(row, vocab_real, temperature, target, ref_logp, lse, grad_ref,
                                               policy_logp, support, grad_policy, R);
    const uint64_t mask = __ballot(live);
    if (lane == 0) count[buf][wave] = __popcll(mask);
    __syncthreads();  // the other buffer is written only after the next one
    int p = before + __popcll(mask & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < kRowThreads / 64; ++w) {
      const int c = count[buf][w];
      if (w < wave) p += c;
      before += c;
    }
    if (live) {
      coef[p] = R;
      row_of[p] = static_cast<int32_t>(row);
    }
    if (row < n_rows) place[row] = live ? p : -1;
  }
  if (threadIdx.x == 0) *n_act = before;
}

// One wave a row: a row with a gradient is copied to its place, another one's
// grad_hidden (when wanted; `bytes` a row) is set to zeros.
__global__ __launch_bounds__(256) void k_gather(const uint16_t* __restrict__ h, int64_t n_rows, int d, int64_t ldh,
                                                const int32_t* __restrict__ place, uint16_t* __restrict__ to,
                                                uint8_t* __restrict__ gh, int64_t gh_stride_bytes, int gh_bytes) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= n_rows) return;  // uniform across the wave
  const int p = place[row];
  if (p >= 0) {
    const u32x4* __restrict__ src = reinterpret_cast<const u32x4*>(h + row * ldh);
    u32x4* __restrict__ dst = reinterpret_cast<u32x4*>(to + static_cast<int64_t>(p) * d);
    for (int v = lane; v < d / 8; v += 64) dst[v] = src[v];
  } else if (gh) {
    u32x4* __restrict__ dst = reinterpret_cast<u32x4*>(gh + row * gh_stride_bytes);
    for (int v = lane; v < gh_bytes / 16; v += 64) dst[v] = u32x4{0u, 0u, 0u, 0u};
  }
}

// Tiles, with LDS for one workgroup a compute unit (three of Short). Large has the
// largest wave part that the 512 registers hold, so the fewest LDS reads for a
// multiplication; the smaller ones are for products whose Large tiles would leave
// compute units idle.
using Large = Shape<256, 256, 2, 2, 5, 1>;
using Half = Shape<128, 256, 2, 2, 6, 1>;
using Quarter = Shape<128, 128, 2, 2, 9, 1>;
using Few = Shape<64, 128, 2, 2, 12, 1>;
using Short = Shape<128, 128, 2, 2, 3, 3>;  // sums over few rows: bound by their stores, three tiles at a time

constexpr int kTile = 256;  // columns of G are padded to whole tiles

enum Pass { kLogits = 0, kHidden = 1, kWeight = 2 };

// Where the sums of grad_hidden go that are made one shard after another: the buffers
// `add` in order in front of them, then float32 sums of the rows with a gradient, or
// (row_of given) the output's rows.
struct HiddenOut {
  const float* add[3];  // [rows with a gradient x d]
  int n_add;
  int type;
  void* out;
  int64_t ldo;
  const int32_t* row_of;
};

struct Args {
  const uint16_t* h;   // gathered hidden states [n_act x d]
  const uint16_t* w;   // projection rows of the launch's first shard
  uint16_t* g;         // G [shard of the launch][n_cap x ldg]
  int64_t ldw;
  int64_t ldg;
  int64_t g_step;      // values between shards of G
  const int32_t* n_act;
  const RowCoef* coef;
  int64_t col0;        // first (global) column of the launch
  int64_t cols;        // its real columns
  int full, rest;      // whole shards of them, columns of the next
  int width;           // columns of a shard
  int shards;          // shards of the launch
  int d;
  int in_turn;         // grad_hidden may be summed one shard after another:
  int turn;            //   then this launch is for shard `turn`
  HiddenOut hid;       //   and its sums go here; else all shards' go to
  float* parts;        // [shard of the launch][part_step]
  int64_t part_step;
  void* gw;            // grad_weight at the launch's first column
  int64_t ldgw;
};

// Shard, tile and sizes of tile u of a launch.
struct Where {
  int shard, m, n, cols;
};

// Tiles of a product over n rows with a gradient (`shards` of them in kHidden, a
// shard without real columns among them: it has its empty sums all the same).
template <class S, Pass kPass>
__host__ __device__ __forceinline__ int tile_count(const Args& a, int n, int shards) {
  const int mt = (n + S::BM - 1) / S::BM;
  const int dt = (a.d + S::BN - 1) / S::BN;
  if (kPass == kHidden) return mt * dt * shards;
  constexpr int v = kPass == kWeight ? S::BM : S::BN;
  return (kPass == kLogits ? mt : dt) * (a.full * ((a.width + v - 1) / v) + (a.rest + v - 1) / v);
}

// The tiles of a product, taken on the device for the rows that have a gradient: of
// one kind (0 .. 3: Large, Half, Quarter, Few), or whole rounds of Large tiles and what
// is left of them cut into smaller ones. Whichever has the least rounds over the compute
// units times a round's cost; the larger kind where that is equal (64 rows of the 151936
// x 4096 head: logits and grad_hidden 527 us, with Large logits 604; 128 rows 675 and
// 705; 640 rows with Large 1635, with Few 2527, with Large's last rounds cut 1520).
// Costs: of a tile's slice in hundredths of Large's, from the logits of 1500 rows and
// 76000 columns at 4096 (Large 868 us for 1800 tiles, 8 rounds; Half 1121 for 3600,
// 15; Quarter 1279 for 7152, 28).
struct Choice {
  int kind, cost;
  int whole;  // Large tiles that come first
};

template <Pass kPass>
__host__ __device__ __forceinline__ Choice tiles_for(const Args& a, int n, int shards) {
  constexpr int kUnits = 256;
  const auto rounds = [](int tiles) { return (tiles + kUnits - 1) / kUnits; };
  const int large = tile_count<Large, kPass>(a, n, shards);
  const int whole = large / kUnits, rest = large % kUnits;
  Choice best{0, rounds(large) * 100, 0};
  const auto look = [&](int kind, int cost, int tiles, int parts) {
    if (rounds(tiles) * cost < best.cost) best = Choice{kind, rounds(tiles) * cost, 0};
    const int mixed = whole * 100 + rounds(rest * parts) * cost;
    if (whole > 0 && mixed < best.cost) best = Choice{kind, mixed, whole * kUnits};
  };
  look(1, 70, tile_count<Half, kPass>(a, n, shards), 2);
  look(2, 44, tile_count<Quarter, kPass>(a, n, shards), 4);
  look(3, 30, tile_count<Few, kPass>(a, n, shards), 8);
  return best;
}

// Whether grad_hidden's shards are summed one after another, each added to the ones
// before as it ends: where that takes no longer than all at once, which writes and
// reads a partial sum for every shard (8192 rows of the 151936 x 4096 head: 15.5 ms
// with the logits, all at once 15.9).
__host__ __device__ __forceinline__ bool one_by_one(const Args& a, int n) {
  return tiles_for<kHidden>(a, n, 1).cost * a.shards <= tiles_for<kHidden>(a, n, a.shards).cost;
}

template <class S, Pass kPass>
__device__ __forceinline__ Where where_is(const Args& a, int n_act, int first, int u) {
  const int mt = (n_act + S::BM - 1) / S::BM;
  const int dt = (a.d + S::BN - 1) / S::BN;
  constexpr int cols = kPass == kWeight ? S::BM : S::BN;
  const int per = (a.width + cols - 1) / cols;
  const int each = kPass == kHidden ? mt * dt : (kPass == kLogits ? mt : dt) * per;
  Where w;
  w.shard = u / each + first;
  const int64_t left = a.cols - static_cast<int64_t>(w.shard) * a.width;
  w.cols = static_cast<int>(left < 0 ? 0 : (left < a.width ? left : a.width));
  const int v = u % each;
  const int vt = (w.cols + cols - 1) / cols;
  if (kPass == kLogits) tile_at(v, mt, vt, w.m, w.n);
  if (kPass == kHidden) tile_at(v, mt, dt, w.m, w.n);
  if (kPass == kWeight) tile_at(v, vt, dt, w.m, w.n);
  return w;
}

// Which tiles a walk goes through: those of its kind, or with `cut` its kind's parts of
// the Large tiles from `from` on (a part may lie past the last row or column: it is a
// sum of zeros, and is not stored).
struct Walk {
  bool cut;
  int from;   // Large tile of the first part
  int shard;  // kHidden one by one: every tile is of this shard
  int count;
};

template <class S, Pass kPass>
__device__ __forceinline__ Where where_is(const Args& a, int n_act, const Walk& walk, int u) {
  constexpr int kM = Large::BM / S::BM, kN = Large::BN / S::BN;
  if (kM * kN == 1 || !walk.cut) return where_is<S, kPass>(a, n_act, walk.shard, u);  // uniform
  Where w = where_is<Large, kPass>(a, n_act, walk.shard, walk.from + u / (kM * kN));
  const int part = u % (kM * kN);
  w.m = w.m * kM + part % kM;
  w.n = w.n * kN + part / kM;
  return w;
}

template <class S, Pass kPass>
__device__ __forceinline__ TileIn tile_in(const Args& a, int n_act, const Where& w) {
  TileIn t;
  const uint16_t* wp = a.w + static_cast<int64_t>(w.shard) * a.width * a.ldw;
  const uint16_t* gp = a.g + w.shard * a.g_step;
  const int rows = n_act - w.m * S::BM < S::BM ? n_act - w.m * S::BM : S::BM;
  if (kPass == kLogits) {
    const int vr = w.cols - w.n * S::BN < S::BN ? w.cols - w.n * S::BN : S::BN;  // (below 1: none)
    t.k_end = a.d;
    t.a = panel_rows(a.h + static_cast<int64_t>(w.m) * S::BM * a.d, rows, a.d, a.d);
    t.b = panel_rows(wp + static_cast<int64_t>(w.n) * S::BN * a.ldw, vr, static_cast<int>(a.ldw), a.d);
  } else if (kPass == kHidden) {
    t.k_end = w.cols;
    // G is zero up to whole slices (an odd end would cut the last row's last word off)
    const int k = w.cols > 0 ? slices_of(w.cols) * kSlice : 0;
    t.a = panel_rows(gp + static_cast<int64_t>(w.m) * S::BM * a.ldg, rows, static_cast<int>(a.ldg), k);
    t.b = panel_cols(wp + w.n * S::BN, a.d - w.n * S::BN, S::BN);
  } else {
    t.k_end = n_act;
    t.a = panel_cols(gp + w.m * S::BM, a.ldg - w.m * S::BM, S::BM);
    t.b = panel_cols(a.h + w.n * S::BN, a.d - w.n * S::BN, S::BN);
  }
  return t;
}

// Two neighbouring blocks' 32 columns of a row in BF16: this lane's 8, at column
// 16 (h % 2) + 8 (h / 2) of the pair, h = lane / 16 (the even quarters of the wave
// give their part of the second block for the odd ones' part of the first).
__device__ __forceinline__ u32x4 pair_words(const f32x4& x, const f32x4& y) {
  const auto lo = __builtin_amdgcn_permlane16_swap(rlk::pack_bf16(x.x, x.y), rlk::pack_bf16(y.x, y.y), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(rlk::pack_bf16(x.z, x.w), rlk::pack_bf16(y.z, y.w), false, false);
  return u32x4{lo[0], hi[0], lo[1], hi[1]};
}
__device__ __forceinline__ int pair_column(int h) { return 16 * (h & 1) + 8 * (h >> 1); }

// The lane, formed where it stands: what is derived from it in an epilogue is not
// kept in registers through the tile's loop.
__device__ __forceinline__ int lane_here() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// G of the tile from its sums: BF16 logits (rounded to nearest even), the
// gradient formula, BF16 again: the matrix cores' operand in both products that follow
// (two BF16 parts would double them), of the type and bits of rlk_logp_backward. Each G is off
// by at most 2^-8 of itself and 1.7e-3 as a root mean square, BF16 outputs by 2.0e-3 to 2.4e-3 of their norm
// in batches (up to 3.4e-3 where few entries of G are large), of which 1.7e-3 is their own rounding.
// Columns past the shard's real ones hold zeros.
template <class S>
__device__ __forceinline__ void store_g(const Args& a, int n_act, const Where& w, const f32x4 (&acc)[S::MB][S::NB]) {
  constexpr int kCols = S::NB * 16;       // of a wave
  const int lane = lane_here();
  const int h = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int wm = wave % S::WM;
  const int wn = wave / S::WM;
  const int cw = w.n * S::BN + wn * kCols;  // first column of the wave's part in the shard
  const bool whole = cw + kCols <= w.cols;
  const int64_t col = a.col0 + static_cast<int64_t>(w.shard) * a.width + cw;
  uint16_t* __restrict__ g = a.g + w.shard * a.g_step;
#pragma unroll
  for (int i = 0; i < S::MB; ++i) {
    const int gr = w.m * S::BM + (wm * S::MB + i) * 16 + (lane & 15);
    const RowCoef R = a.coef[gr < n_act ? gr : 0];
    const bool policy = __any(R.s_p != 0.0f);
    f32x4 v[S::NB];
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
      v[j] = taken(acc[i][j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __uint_as_float(static_cast<uint32_t>(__builtin_bit_cast(
                                            uint16_t, static_cast<__bf16>(v[j][e]))) << 16);
        float o = R.s_r * __builtin_amdgcn_exp2f(fmaf(x, R.c, R.a_r));
        if (policy) {  // uniform
          const float q = x >= R.thr ? __builtin_amdgcn_exp2f(fmaf(x, R.c, R.a_p)) : 0.0f;
          o = o + R.s_p * q;
        }
        v[j][e] = o;
      }
    }
    const int64_t lc = R.target - col;
    const bool tin = R.target >= 0 && lc >= 0 && lc < kCols;
    if (__any(tin)) {
      const int lci = static_cast<int>(tin ? lc : 0);
      const int kt = tin && ((lci >> 2) & 3) == h ? (lci >> 4) * 4 + (lci & 3) : -1;
#pragma unroll
      for (int k = 0; k < 4 * S::NB; ++k) v[k >> 2][k & 3] = k == kt ? R.g_t : v[k >> 2][k & 3];
    }
    if (!whole) {
      const int lim = w.cols - cw - 4 * h;  // this lane's column 16 j + e is real iff below lim
#pragma unroll
      for (int k = 0; k < 4 * S::NB; ++k) v[k >> 2][k & 3] = 16 * (k >> 2) + (k & 3) < lim ? v[k >> 2][k & 3] : 0.0f;
    }
    uint16_t* dst = g + static_cast<int64_t>(gr) * a.ldg + cw + pair_column(h);
#pragma unroll
    for (int j = 0; j < S::NB; j += 2) {
      const u32x4 o = pair_words(v[j], v[j + 1]);
      if (gr < n_act) *reinterpret_cast<u32x4*>(dst + 16 * j) = o;  // ldg is a multiple of 256: the tile's columns exist
    }
  }
}

// Stores blocks (i, j) and (i, j + 1), the lane's row of which starts at out + at.
template <int kType>
__device__ __forceinline__ void store_pair(const f32x4& x, const f32x4& y, bool ok, void* __restrict__ out, int64_t at,
                                           int h) {
  if (kType == RLK_GRAD_BF16) {
    const u32x4 v = pair_words(x, y);
    if (ok) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at + pair_column(h)) = v;
  } else if (ok) {
    f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at + 4 * h);
    dst[0] = kType == RLK_GRAD_F32_ADD ? dst[0] + x : x;
    dst[4] = kType == RLK_GRAD_F32_ADD ? dst[4] + y : y;
  }
}

template <class S, int kType>
__device__ __forceinline__ void store_hidden(const Args& a, int n_act, bool in_turn, const Where& w,
                                             const f32x4 (&acc)[S::MB][S::NB]) {
  const int lane = lane_here();
  const int h = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int wm = wave % S::WM;
  const int wn = wave / S::WM;
  const int cw = w.n * S::BN + wn * S::NB * 16;
  const int n_add = in_turn ? a.hid.n_add : 0;
  const int32_t* row_of = in_turn ? a.hid.row_of : nullptr;
  const int64_t ldo = in_turn ? a.hid.ldo : a.d;
  void* out = in_turn ? a.hid.out : a.parts + w.shard * a.part_step;
#pragma unroll
  for (int i = 0; i < S::MB; ++i) {
    const int gr = w.m * S::BM + (wm * S::MB + i) * 16 + (lane & 15);
    f32x4 v[S::NB];
#pragma unroll
    for (int j = 0; j < S::NB; ++j) v[j] = taken(acc[i][j]);
    for (int k = 0; k < n_add; ++k) {
      const float* from = a.hid.add[k] + static_cast<int64_t>(gr) * a.d + cw + 4 * h;
      f32x4 o[S::NB];
#pragma unroll
      for (int j = 0; j < S::NB; ++j) {
        o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (gr < n_act && cw + 16 * j < a.d) o[j] = *reinterpret_cast<const f32x4*>(from + 16 * j);  // d is a multiple of 64
      }
#pragma unroll
      for (int j = 0; j < S::NB; ++j) v[j] = o[j] + v[j];
    }
    const int64_t row = row_of && gr < n_act ? row_of[gr] : gr;
    const int64_t at = row * ldo + cw;
#pragma unroll
    for (int j = 0; j < S::NB; j += 2)
      store_pair<kType>(v[j], v[j + 1], gr < n_act && cw + 16 * j < a.d, out, at + 16 * j, h);
  }
}

template <class S, int kType>
__device__ __forceinline__ void store_weight(const Args& a, const Where& w, const f32x4 (&acc)[S::MB][S::NB]) {
  const int lane = lane_here();
  const int h = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int wm = wave % S::WM;
  const int wn = wave / S::WM;
  const int cw = w.n * S::BN + wn * S::NB * 16;
  const int64_t first = static_cast<int64_t>(w.shard) * a.width;
#pragma unroll
  for (int i = 0; i < S::MB; ++i) {
    const int v = w.m * S::BM + (wm * S::MB + i) * 16 + (lane & 15);
    const int64_t at = (first + v) * a.ldgw + cw;
#pragma unroll
    for (int j = 0; j < S::NB; j += 2)
      store_pair<kType>(taken(acc[i][j]), taken(acc[i][j + 1]), v < w.cols && cw + 16 * j < a.d, a.gw, at + 16 * j, h);
  }
}

template <class S, Pass kPass, int kType>
__device__ __forceinline__ void product_tiles(const Args& a, int n_act, bool in_turn, const Walk& walk, uint8_t* smem) {
  const int n_tiles = walk.count;
  const int most = (n_tiles + kXcds - 1) / kXcds * kXcds;
  const int grid = static_cast<int>(gridDim.x) < most ? static_cast<int>(gridDim.x) : most;
  if (static_cast<int>(blockIdx.x) >= grid) return;
  int u = first_tile(grid);
  if (u >= n_tiles) return;  // uniform across the workgroup
  int loads = u;  // the tile that the loads come to next
  const auto next = [&](TileIn& t) __attribute__((always_inline)) {
    if (loads >= n_tiles) return false;
    t = tile_in<S, kPass>(a, n_act, where_is<S, kPass>(a, n_act, walk, loads));
    loads += grid;
    return true;
  };
  Tiles<S, kPass == kWeight, kPass != kLogits, decltype(next)> tiles(
      next, smem, kPass == kLogits ? a.d : static_cast<int>(a.ldg), kPass == kWeight ? a.d : static_cast<int>(a.ldw));
  tiles.start();
  for (; u < n_tiles; u += grid) {
    const Where w = where_is<S, kPass>(a, n_act, walk, u);
    f32x4 acc[S::MB][S::NB];
    tiles.sums(acc, slices_of(kPass == kLogits ? a.d : (kPass == kHidden ? w.cols : n_act)));
    if (kPass == kLogits) store_g<S>(a, n_act, w, acc);
    if (kPass == kHidden) store_hidden<S, kType>(a, n_act, in_turn, w, acc);
    if (kPass == kWeight) store_weight<S, kType>(a, w, acc);
  }
}

// kLogits and kHidden, on the tiles that suit the rows with a gradient.
template <Pass kPass, int kType>
__global__ __launch_bounds__(kThreads, 1) void k_product(Args a) {
  static_assert(Large::kLds >= Half::kLds && Large::kLds >= Quarter::kLds && Large::kLds >= Few::kLds, "LDS of each kind");
  __shared__ __attribute__((aligned(16))) uint8_t smem[Large::kLds];
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  const bool in_turn = kPass == kHidden && a.in_turn && one_by_one(a, n_act);
  if (kPass == kHidden && !in_turn && a.turn > 0) return;  // the first launch has summed all shards
  const int shards = in_turn ? 1 : a.shards;
  const Choice best = tiles_for<kPass>(a, n_act, shards);
  int kind = best.whole > 0 ? 0 : best.kind;
  int done = 0;  // Large tiles before the walk at hand
#pragma unroll 1
  for (;;) {
    Walk walk{done > 0, done, in_turn ? a.turn : 0, 0};
    if (kind == 0) {
      walk.count = best.whole > 0 ? best.whole : tile_count<Large, kPass>(a, n_act, shards);
      product_tiles<Large, kPass, kType>(a, n_act, in_turn, walk, smem);
    } else {
      const int rest = tile_count<Large, kPass>(a, n_act, shards) - done;
      if (kind == 1) {
        walk.count = walk.cut ? rest * 2 : tile_count<Half, kPass>(a, n_act, shards);
        product_tiles<Half, kPass, kType>(a, n_act, in_turn, walk, smem);
      } else if (kind == 2) {
        walk.count = walk.cut ? rest * 4 : tile_count<Quarter, kPass>(a, n_act, shards);
        product_tiles<Quarter, kPass, kType>(a, n_act, in_turn, walk, smem);
      } else {
        walk.count = walk.cut ? rest * 8 : tile_count<Few, kPass>(a, n_act, shards);
        product_tiles<Few, kPass, kType>(a, n_act, in_turn, walk, smem);
      }
    }
    if (done == best.whole) return;  // uniform: there is no second walk, or it is over
    done = best.whole;
    kind = best.kind;
    // no load of the first walk (of zeros, past its last tile) comes after this
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

template <class S, int kType>
__global__ __launch_bounds__(kThreads, S::kPer) void k_weight(Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  product_tiles<S, kWeight, kType>(a, n_act, false, Walk{false, 0, 0, tile_count<S, kWeight>(a, n_act, a.shards)}, smem);
}

// The fixed sum of `count` (1, 2, 4 or 8) partial sums, neighbours first.
template <typename F>
__device__ __forceinline__ f32x4 tree(int count, const F& part) {
  f32x4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < count) v[k] = part(k);
#pragma unroll
  for (int s = 1; s < 8; s *= 2)
#pragma unroll
    for (int k = 0; k + s < 8; k += 2 * s)
      if (s < count && k < count) v[k] = v[k] + v[k + s];
  return v[0];
}

__device__ __forceinline__ void store4(void* out, int type, int64_t at, const f32x4& v) {
  if (type == RLK_GRAD_BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(rlk::pack_bf16(v.x, v.y),
                                                                            rlk::pack_bf16(v.z, v.w));
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = v;
}

// Row r of the rows with a gradient: the partial sums of a launch's shards, then the
// earlier ones.
__global__ __launch_bounds__(256) void k_combine(Args a, HiddenOut o) {
  const int n = *a.n_act;
  if (a.in_turn && one_by_one(a, n)) return;  // done already
  const int64_t vecs = static_cast<int64_t>(n) * (a.d / 4);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < vecs;
       v += static_cast<int64_t>(gridDim.x) * 256) {
    f32x4 s = tree(a.shards, [&](int k) { return *reinterpret_cast<const f32x4*>(a.parts + k * a.part_step + v * 4); });
    for (int k = 0; k < o.n_add; ++k) s = *reinterpret_cast<const f32x4*>(o.add[k] + v * 4) + s;
    const int64_t r = v / (a.d / 4);
    const int64_t c = (v - r * (a.d / 4)) * 4;
    store4(o.out, o.type, (o.row_of ? o.row_of[r] : r) * o.ldo + c, s);
  }
}

__global__ __launch_bounds__(256) void k_merge(const float* __restrict__ parts, int64_t step, int count,
                                               int64_t n_rows, int d, void* __restrict__ out, int64_t ldo, int type) {
  const int64_t vecs = n_rows * (d / 4);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < vecs;
       v += static_cast<int64_t>(gridDim.x) * 256) {
    const f32x4 s = tree(count, [&](int k) { return *reinterpret_cast<const f32x4*>(parts + k * step + v * 4); });
    const int64_t r = v / (d / 4);
    store4(out, type, r * ldo + (v - r * (d / 4)) * 4, s);
  }
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static int32_t launched() { return hipGetLastError() == hipSuccess ? RLK_OK : RLK_ERR_HIP; }

static int32_t check_shapes(int64_t n_rows, int64_t d, const rlk_vocab_layout* L) {
  if (L == nullptr) return RLK_ERR_NULL;
  if (n_rows < 0 || n_rows > kMaxRows) return RLK_ERR_SHAPE;
  if (L->n_shards != kShards) return RLK_ERR_SHAPE;
  if (L->vocab_padded < 64 || L->vocab_padded > kMaxVocab || L->vocab_padded % 64 != 0) return RLK_ERR_SHAPE;
  if (L->vocab_real < 1 || L->vocab_real > L->vocab_padded) return RLK_ERR_SHAPE;
  if (L->row_stride < L->vocab_padded || L->row_stride % 8 != 0) return RLK_ERR_SHAPE;
  if (!(L->groups == 1 || L->groups == 2 || L->groups == 4 || L->groups == 8)) return RLK_ERR_GROUPS;
  if (d < 64 || d > kMaxD || d % 64 != 0) return RLK_ERR_SHAPE;
  return RLK_OK;
}

static bool stride_ok(int64_t ld, int64_t d) { return ld >= d && ld % 8 == 0 && ld <= kMaxLd; }

// The workspace and how many shards of G it holds at a time.
struct Plan {
  int width;        // columns of a shard
  int local;        // the rank's shards
  int at_once;      // shards of a launch (1, 2, 4 or 8)
  int64_t ldg;
  int64_t g_step;
  int64_t part_step;
  int n_parts;      // partial sums of grad_hidden: of a launch's shards, and earlier ones that wait
  size_t n_act, coef, row_of, place, h, g, parts, bytes;
};

// G of one launch may take this much when it takes more than one shard.
constexpr int64_t kGBudget = int64_t(640) << 20;

static Plan plan_for(int64_t n_rows, int64_t d, const rlk_vocab_layout* L) {
  Plan p;
  p.width = static_cast<int>(L->vocab_padded / kShards);
  p.local = kShards / L->groups;
  p.ldg = (static_cast<int64_t>(p.width) + kTile - 1) / kTile * kTile;
  p.g_step = n_rows * p.ldg;
  p.part_step = n_rows * d;
  p.at_once = p.local;
  while (p.at_once > 1 && p.at_once * p.g_step * 2 > kGBudget) p.at_once /= 2;
  int levels = 0;  // sums that wait for their neighbours
  for (int k = p.local / p.at_once; k > 1; k /= 2) ++levels;
  p.n_parts = (p.at_once > 1 ? p.at_once : 0) + levels;  // (shard by shard: at most as many)
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.n_act = take(sizeof(int32_t));
  p.coef = take(static_cast<size_t>(n_rows) * sizeof(RowCoef));
  p.row_of = take(static_cast<size_t>(n_rows) * sizeof(int32_t));
  p.place = take(static_cast<size_t>(n_rows) * sizeof(int32_t));
  p.h = take(static_cast<size_t>(n_rows) * d * 2);
  p.g = take(static_cast<size_t>(p.at_once) * p.g_step * 2);
  p.parts = take(static_cast<size_t>(p.n_parts) * p.part_step * 4);
  p.bytes = at;
  return p;
}

// Bytes for n_rows rows and for any fewer: where a launch takes fewer shards from
// some row count on, the rows just below it need more.
static size_t bytes_for(int64_t n_rows, int64_t d, const rlk_vocab_layout* L) {
  size_t most = plan_for(n_rows, d, L).bytes;
  const int64_t ldg = plan_for(0, d, L).ldg;
  for (int a = kShards / L->groups; a > 1; a /= 2) {
    const int64_t n = kGBudget / (a * ldg * 2);  // the most rows with `a` shards at once
    if (n < n_rows) {
      const size_t b = plan_for(n, d, L).bytes;
      most = b > most ? b : most;
    }
  }
  return most;
}

// Compute units of the current device (cached per device), a multiple of 8.
static int cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return 256;
  n = (n + kXcds - 1) / kXcds * kXcds;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// (The rows with a gradient are counted on the device: n_rows is the most.)
static dim3 grid_for(int tiles, int per) {
  const int most = cu_count() * per;
  const int want = (tiles + kXcds - 1) / kXcds * kXcds;
  return dim3(static_cast<unsigned>(want < most ? want : most));
}

template <Pass kPass, int kType>
static int32_t product(const Args& a, int64_t n_rows, hipStream_t stream) {
  const int n = static_cast<int>(n_rows);  // Few has the most tiles
  k_product<kPass, kType><<<grid_for(tile_count<Few, kPass>(a, n, a.shards), 1), dim3(kThreads), 0, stream>>>(a);
  return launched();
}

// Short tiles for few rows and few tiles (64 rows of an 8000 x 512 head 33 us a call,
// with Large 37; 77 of 50021 x 1088, 1000 Large tiles, 103 and 106), Large ones
// otherwise (64 rows of 151936 x 4096, 9500 tiles: 630 us with the logits, with Short
// 682; 128 rows 737 and 829; 256 rows 930 and 1065). The host chooses, by all rows; a small
// head with many rows gets few Large tiles (8000 x 512: 64 for 256 compute units), which the
// other products' choice by rounds would cut.
template <int kType>
static int32_t weight_product(const Args& a, int64_t n_rows, hipStream_t stream) {
  const int n = static_cast<int>(n_rows);
  const int tiles = tile_count<Large, kWeight>(a, n, a.shards);
  if (n <= 128 && tiles <= 1024)
    k_weight<Short, kType><<<grid_for(tile_count<Short, kWeight>(a, n, a.shards), Short::kPer), dim3(kThreads), 0, stream>>>(a);
  else
    k_weight<Large, kType><<<grid_for(tiles, 1), dim3(kThreads), 0, stream>>>(a);
  return launched();
}

static unsigned vec_grid(int64_t vecs) {
  const int64_t blocks = (vecs + 255) / 256;
  return static_cast<unsigned>(blocks < 1 ? 1 : (blocks < 4096 ? blocks : 4096));
}

}  // namespace rlk_lin_grad

extern "C" {

size_t rlk_linear_logp_backward_workspace_bytes(int64_t n_rows, int64_t d_model, const rlk_vocab_layout* layout) {
  using namespace rlk_lin_grad;
  if (check_shapes(n_rows, d_model, layout) != RLK_OK) return 0;
  return bytes_for(n_rows, d_model, layout);
}

int32_t rlk_linear_logp_backward(const uint16_t* hidden, int64_t n_rows, int64_t d_model, int64_t hidden_stride,
                                 const uint16_t* weight, int64_t weight_stride, const rlk_vocab_layout* layout,
                                 int32_t rank, const float* temperature, const int64_t* target,
                                 const float* ref_logp, const float* lse, const float* grad_ref,
                                 const float* policy_logp, const rlk_support_state* support,
                                 const float* grad_policy, void* grad_hidden, int64_t grad_hidden_stride,
                                 int32_t grad_hidden_type, void* grad_weight, int64_t grad_weight_stride,
                                 int32_t grad_weight_type, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  using namespace rlk_lin_grad;
  int32_t st = check_shapes(n_rows, d_model, layout);
  if (st != RLK_OK) return st;
  const int64_t d = d_model;
  if (!stride_ok(hidden_stride, d) || !stride_ok(weight_stride, d)) return RLK_ERR_SHAPE;
  if (rank < 0 || rank >= layout->groups) return RLK_ERR_SHAPE;
  if (!grad_hidden && !grad_weight) return RLK_ERR_NULL;
  if (grad_hidden && (!stride_ok(grad_hidden_stride, d) ||
                      !(grad_hidden_type == RLK_GRAD_BF16 || grad_hidden_type == RLK_GRAD_F32)))
    return RLK_ERR_SHAPE;
  if (grad_weight && (!stride_ok(grad_weight_stride, d) || grad_weight_type < RLK_GRAD_BF16 ||
                      grad_weight_type > RLK_GRAD_F32_ADD))
    return RLK_ERR_SHAPE;
  if (n_rows > 0) {
    if (!hidden || !weight || !temperature || !target) return RLK_ERR_NULL;
    if (!grad_ref && !grad_policy) return RLK_ERR_NULL;
    if (grad_ref && (!ref_logp || !lse)) return RLK_ERR_NULL;
    if (grad_policy && (!policy_logp || !support)) return RLK_ERR_NULL;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(temperature, 4) || !aligned(target, 8) ||
        !aligned(ref_logp, 4) || !aligned(lse, 4) || !aligned(grad_ref, 4) || !aligned(policy_logp, 4) ||
        !aligned(support, 4) || !aligned(grad_policy, 4))
      return RLK_ERR_ALIGN;
  }
  if (!workspace) return RLK_ERR_NULL;
  if (!aligned(workspace, 16) || !aligned(grad_hidden, 16) || !aligned(grad_weight, 16)) return RLK_ERR_ALIGN;
  if (workspace_bytes < bytes_for(n_rows, d, layout)) return RLK_ERR_WORKSPACE;
  const Plan p = plan_for(n_rows, d, layout);

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* n_act = reinterpret_cast<int32_t*>(ws + p.n_act);
  RowCoef* coef = reinterpret_cast<RowCoef*>(ws + p.coef);
  int32_t* row_of = reinterpret_cast<int32_t*>(ws + p.row_of);
  int32_t* place = reinterpret_cast<int32_t*>(ws + p.place);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + p.h);
  float* parts = reinterpret_cast<float*>(ws + p.parts);
  if (n_rows == 0 && (!grad_weight || grad_weight_type == RLK_GRAD_F32_ADD)) return RLK_OK;
  k_rows<<<dim3(1), dim3(kRowThreads), 0, stream>>>(n_rows, layout->vocab_real, temperature, target, ref_logp, lse,
                                                     grad_ref, policy_logp, support, grad_policy, coef, row_of, place,
                                                     n_act);
  if ((st = launched()) != RLK_OK) return st;
  if (n_rows > 0) {
    const int size = grad_hidden_type == RLK_GRAD_BF16 ? 2 : 4;
    k_gather<<<dim3(static_cast<unsigned>((n_rows + 3) / 4)), dim3(256), 0, stream>>>(
        hidden, n_rows, static_cast<int>(d), hidden_stride, place, h, static_cast<uint8_t*>(grad_hidden),
        grad_hidden_stride * size, static_cast<int>(d) * size);
    if ((st = launched()) != RLK_OK) return st;
  }

  const int64_t first = static_cast<int64_t>(rank) * p.local * p.width;  // the rank's first column
  Args a{};
  a.h = h;
  a.g = reinterpret_cast<uint16_t*>(ws + p.g);
  a.ldw = weight_stride;
  a.ldg = p.ldg;
  a.g_step = p.g_step;
  a.n_act = n_act;
  a.coef = coef;
  a.width = p.width;
  a.d = static_cast<int>(d);
  a.ldgw = grad_weight_stride;
  a.shards = p.at_once;
  a.parts = parts;
  a.part_step = p.part_step;
  a.in_turn = one_by_one(a, static_cast<int>(n_rows));
  for (int s = 0; s < p.local; s += p.at_once) {
    const int64_t c0 = static_cast<int64_t>(s) * p.width;  // columns counted from the rank's first
    const int64_t left = layout->vocab_real - first - c0;
    const int64_t most = static_cast<int64_t>(p.at_once) * p.width;
    a.col0 = first + c0;
    a.cols = left < 0 ? 0 : (left < most ? left : most);
    a.full = static_cast<int>(a.cols / p.width);
    a.rest = static_cast<int>(a.cols % p.width);
    a.w = n_rows > 0 && a.cols > 0 ? weight + c0 * weight_stride : weight;
    if (n_rows > 0 && a.cols > 0) {
      if ((st = product<kLogits, RLK_GRAD_BF16>(a, n_rows, stream)) != RLK_OK) return st;
    }
    if (grad_hidden && n_rows > 0) {
      // The k-th of the sums (of a shard, or of a launch's shards): those of whole
      // pairs, fours and eights wait and are added as their neighbours end. Only one of
      // the two ways is gone, on the device, so both may use the same buffers.
      const auto sum_to = [&](float* waiting, int k, bool last) {
        HiddenOut o{};
        int level = 0;
        for (; (k >> level) & 1; ++level) o.add[level] = waiting + level * p.part_step;
        o.n_add = level;
        o.out = last ? grad_hidden : waiting + level * p.part_step;
        o.ldo = last ? grad_hidden_stride : d;
        o.type = last ? grad_hidden_type : RLK_GRAD_F32;
        o.row_of = last ? row_of : nullptr;
        return o;
      };
      for (a.turn = 0; a.turn < (a.in_turn ? p.at_once : 1); ++a.turn) {
        const int k = s + a.turn;
        a.hid = sum_to(parts, k, k + 1 == p.local);
        // (BF16 is the last shard's, whose launch sums no others unless it is the only one)
        st = a.in_turn && a.hid.type == RLK_GRAD_BF16 ? product<kHidden, RLK_GRAD_BF16>(a, n_rows, stream)
                                                      : product<kHidden, RLK_GRAD_F32>(a, n_rows, stream);
        if (st != RLK_OK) return st;
      }
      a.turn = 0;
      if (p.at_once > 1) {
        k_combine<<<dim3(vec_grid(n_rows * (d / 4))), dim3(256), 0, stream>>>(
            a, sum_to(parts + p.at_once * p.part_step, s / p.at_once, s + p.at_once == p.local));
        if ((st = launched()) != RLK_OK) return st;
      }
    }
    if (grad_weight && a.cols > 0) {
      const int64_t size = grad_weight_type == RLK_GRAD_BF16 ? 2 : 4;
      a.gw = static_cast<uint8_t*>(grad_weight) + c0 * grad_weight_stride * size;
      if (grad_weight_type == RLK_GRAD_BF16)
        st = weight_product<RLK_GRAD_BF16>(a, n_rows, stream);
      else if (grad_weight_type == RLK_GRAD_F32)
        st = weight_product<RLK_GRAD_F32>(a, n_rows, stream);
      else
        st = weight_product<RLK_GRAD_F32_ADD>(a, n_rows, stream);
      if (st != RLK_OK) return st;
    }
  }
  return RLK_OK;
}

int32_t rlk_linear_logp_backward_merge(const float* parts, int64_t part_stride, int32_t groups, int64_t n_rows,
                                       int64_t d_model, void* grad_hidden, int64_t grad_hidden_stride,
                                       int32_t grad_hidden_type, hipStream_t stream) {
  using namespace rlk_lin_grad;
  if (!(groups == 1 || groups == 2 || groups == 4 || groups == 8)) return RLK_ERR_GROUPS;
  if (n_rows < 0 || n_rows > kMaxRows || d_model < 64 || d_model > kMaxD || d_model % 64 != 0) return RLK_ERR_SHAPE;
  if (part_stride < n_rows * d_model || part_stride % 4 != 0 || part_stride > INT64_MAX / 64) return RLK_ERR_SHAPE;
  if (!stride_ok(grad_hidden_stride, d_model) ||
      !(grad_hidden_type == RLK_GRAD_BF16 || grad_hidden_type == RLK_GRAD_F32))
    return RLK_ERR_SHAPE;
  if (n_rows == 0) return RLK_OK;
  if (!parts || !grad_hidden) return RLK_ERR_NULL;
  if (!aligned(parts, 16) || !aligned(grad_hidden, 16)) return RLK_ERR_ALIGN;
  k_merge<<<dim3(vec_grid(n_rows * (d_model / 4))), dim3(256), 0, stream>>>(
      parts, part_stride, groups, n_rows, static_cast<int>(d_model), grad_hidden, grad_hidden_stride,
      grad_hidden_type);
  return launched();
}

}  // extern "C"
