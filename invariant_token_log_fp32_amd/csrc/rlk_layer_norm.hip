// Layer norm / RMS norm in front of the LM head, its backward pass, and the C
// ABI declared in include/rlk_layer_norm.h.
//
// Kernels:
//   k_norm           a workgroup of just the waves that hold a row in registers
//                    (16 or 32 values a thread) goes through rows, the next row's loads
//                    in flight while it reduces one; the weight stays in
//                    registers. Mean and variance are two sums over the values
//                    in registers, so the variance has no cancellation.
//   k_norm_backward  the same walk over rows of x and dy; a thread owns its
//                    columns, so dweight and dbias are summed over the
//                    workgroup's rows in registers and written once
//   k_norm_sums      the workgroups' sums added up, in a fixed tree
//   k_norm_backward_few  both for few rows, in one launch
// All are bound by memory, one pass over the rows: 8192 x 4096 in float32 31 us on the
// GPU (6.4 TB/s), its BF16 backward 34 us and the sums 5, the backward of 65536 x 4096
// 280 us (5.8 TB/s; a large copy reaches 4.9). Small calls are bound by the launch (1 x
// 4096 2.5 us on the GPU).
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "bf16_store.hpp"
#include "logp_device.hpp"
#include "rlk_layer_norm.h"
#include "rlk_logp.h"

namespace rlk_norm_layer {

using rlk::u32x4;

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxLd = int64_t(1) << 21;
constexpr int kMaxD = 16384;
constexpr int kMaxThreads = 512;
constexpr int kMaxWaves = kMaxThreads / 64;
constexpr int kUnits = 256;     // compute units the walk is cut for (a fixed number: the order of the sums depends on it)

// 8 values as they lie in memory.
template <int kType>
struct Raw;
template <>
struct Raw<RLK_TYPE_BF16> {
  u32x4 v;
};
template <>
struct Raw<RLK_TYPE_F32> {
  f32x4 lo, hi;
};

template <int kType>
__device__ __forceinline__ Raw<kType> load8(const void* p, int64_t at) {
  Raw<kType> r;
  if constexpr (kType == RLK_TYPE_BF16) {
    r.v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    r.lo = q[0];
    r.hi = q[1];
  }
  return r;
}

template <int kType>
__device__ __forceinline__ Raw<kType> zero8() {
  Raw<kType> r;
  if constexpr (kType == RLK_TYPE_BF16) {
    r.v = u32x4{0u, 0u, 0u, 0u};
  } else {
    r.lo = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    r.hi = r.lo;
  }
  return r;
}

template <int kType>
__device__ __forceinline__ void widen(const Raw<kType>& r, float (&x)[8]) {
  if constexpr (kType == RLK_TYPE_BF16) {
    rlk::unpack8(r.v, x);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = r.lo[e];
      x[4 + e] = r.hi[e];
    }
  }
}

template <int kType>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  if constexpr (kType == RLK_TYPE_BF16) {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at) =
        u32x4{rlk::pack_bf16(x[0], x[1]), rlk::pack_bf16(x[2], x[3]), rlk::pack_bf16(x[4], x[5]),
              rlk::pack_bf16(x[6], x[7])};
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    q[0] = f32x4{x[0], x[1], x[2], x[3]};
    q[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
}

__device__ __forceinline__ float sum8(const float (&x)[8]) {
  return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

// Sum of two values over the workgroup, the same bits in every thread: over the
// wave by a butterfly, over the waves in order. `turn` alternates between two
// halves of `part`, so one barrier a sum is enough.
__device__ __forceinline__ float2 sum_over(float a, float b, int waves, float2 (&part)[2][kMaxWaves], int turn) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    a = a + __shfl_xor(a, o);
    b = b + __shfl_xor(b, o);
  }
  if (waves == 1) return make_float2(a, b);
  if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  float2 s = part[turn][0];
  for (int w = 1; w < waves; ++w) {
    s.x = s.x + part[turn][w].x;
    s.y = s.y + part[turn][w].y;
  }
  return s;
}

template <int kX, int kW, int kVecs, int kBound>
__global__ __launch_bounds__(kBound) void k_norm(const void* x, int64_t n_rows, int d, int64_t ldx,
                                                 const void* __restrict__ weight, const void* __restrict__ bias,
                                                 int rms, float eps, uint16_t* y, int64_t ldy,
                                                 float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float2 part[2][kMaxWaves];
  const int threads = static_cast<int>(blockDim.x);
  const int waves = threads >> 6;
  const float count = static_cast<float>(d);
  int at[kVecs];
  bool in[kVecs];
  Raw<kW> w[kVecs], b[kVecs];
  Raw<kX> raw[kVecs];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    at[v] = (static_cast<int>(threadIdx.x) + v * threads) * 8;
    in[v] = at[v] < d;
    raw[v] = in[v] ? load8<kX>(x, row * ldx + at[v]) : zero8<kX>();
  }
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    w[v] = in[v] ? load8<kW>(weight, at[v]) : zero8<kW>();
    b[v] = in[v] && bias ? load8<kW>(bias, at[v]) : zero8<kW>();
  }
  int turn = 0;
  for (; row < n_rows; row += gridDim.x) {  // uniform across the workgroup
    float f[kVecs][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) widen<kX>(raw[v], f[v]);
    const int64_t next = row + gridDim.x;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (in[v] && next < n_rows) raw[v] = load8<kX>(x, next * ldx + at[v]);
    float m = 0.0f;
    if (!rms) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) s = s + sum8(f[v]);
      m = sum_over(s, 0.0f, waves, part, turn).x / count;
      turn ^= 1;
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[v][e] = in[v] ? f[v][e] - m : 0.0f;
        q[e] = f[v][e] * f[v][e];
      }
      s = s + sum8(q);
    }
    const float r = 1.0f / sqrtf(sum_over(s, 0.0f, waves, part, turn).x / count + eps);
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (in[v]) {
        float o[8], wv[8], bv[8];
        widen<kW>(w[v], wv);
        widen<kW>(b[v], bv);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f[v][e] * r * wv[e] + bv[e];
        store8<RLK_TYPE_BF16>(y, row * ldy + at[v], o);
      }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = m;
      if (rstd_out) rstd_out[row] = r;
    }
  }
}

// A value's part of dweight: nothing where dy is 0, whatever stands there.
__device__ __forceinline__ float weight_term(float dy, float hat) { return dy != 0.0f ? dy * hat : 0.0f; }

// parts: per workgroup d sums of dy * xhat, then (kBias) d sums of dy.
template <int kX, int kW, int kVecs, bool kBias>
__device__ __forceinline__ void backward_rows(const uint16_t* dy, int64_t lddy, const void* x, int64_t n_rows, int d,
                                              int64_t ldx, const void* __restrict__ weight, int rms,
                                              const float* __restrict__ mean, const float* __restrict__ rstd, void* dx,
                                              int64_t lddx, float* __restrict__ parts, int step) {
  __shared__ float2 part[2][kMaxWaves];
  __shared__ int any[2];
  const int threads = static_cast<int>(blockDim.x);
  const int waves = threads >> 6;
  const float count = static_cast<float>(d);
  int at[kVecs];
  bool in[kVecs];
  Raw<kW> w[kVecs];
  float dw[kVecs][8], db[kVecs][8];
  Raw<kX> raw[kVecs];
  Raw<RLK_TYPE_BF16> up[kVecs];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    at[v] = (static_cast<int>(threadIdx.x) + v * threads) * 8;
    in[v] = at[v] < d;
    raw[v] = in[v] ? load8<kX>(x, row * ldx + at[v]) : zero8<kX>();
    up[v] = in[v] ? load8<RLK_TYPE_BF16>(dy, row * lddy + at[v]) : zero8<RLK_TYPE_BF16>();
  }
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    w[v] = in[v] ? load8<kW>(weight, at[v]) : zero8<kW>();
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
  }
  if (threadIdx.x < 2) any[threadIdx.x] = 0;
  __syncthreads();
  int turn = 0;
  for (; row < n_rows; row += step) {  // uniform across the workgroup
    float f[kVecs][8], g[kVecs][8];
    uint32_t some = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      widen<kX>(raw[v], f[v]);
      widen<RLK_TYPE_BF16>(up[v], g[v]);
      some |= (up[v].v.x | up[v].v.y | up[v].v.z | up[v].v.w) & 0x7FFF7FFFu;
    }
    const int64_t next = row + step;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (in[v] && next < n_rows) {
        raw[v] = load8<kX>(x, next * ldx + at[v]);
        up[v] = load8<RLK_TYPE_BF16>(dy, next * lddy + at[v]);
      }
    float r = rstd[row];
    float m = rms ? 0.0f : mean[row];
    // a row without a gradient: zeros, whatever x and the statistics hold
    bool live = __any(some != 0);
    if (waves > 1) {
      if (live && (threadIdx.x & 63) == 0) any[turn] = 1;
      __syncthreads();
      live = any[turn] != 0;
      if (threadIdx.x == 0) any[turn ^ 1] = 0;  // read by all before the barrier of the sums below
    }
    r = live ? r : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float q1[8], q2[8], wv[8];
      widen<kW>(w[v], wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hat = live ? (f[v][e] - m) * r : 0.0f;
        dw[v][e] = dw[v][e] + weight_term(g[v][e], hat);
        if (kBias) db[v][e] = db[v][e] + g[v][e];
        f[v][e] = hat;
        g[v][e] = live ? g[v][e] * wv[e] : 0.0f;  // (0 times a weight that is no number would not be 0)
        q1[e] = g[v][e];
        q2[e] = g[v][e] * hat;
      }
      s1 = s1 + sum8(q1);
      s2 = s2 + sum8(q2);
    }
    const float2 s = sum_over(s1, s2, waves, part, turn);
    turn ^= 1;
    const float c1 = rms ? 0.0f : s.x / count;
    const float c2 = s.y / count;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (in[v] && dx) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = r * (g[v][e] - c1 - f[v][e] * c2);
        store8<kX>(dx, row * lddx + at[v], o);
      }
  }
  if (!parts) return;
#pragma unroll
  for (int v = 0; v < kVecs; ++v)
    if (in[v]) {
      float* p = parts + static_cast<int64_t>(blockIdx.x) * d * (kBias ? 2 : 1) + at[v];
      store8<RLK_TYPE_F32>(p, 0, dw[v]);
      if (kBias) store8<RLK_TYPE_F32>(p, d, db[v]);
    }
}

template <int kX, int kW, int kVecs, bool kBias, int kBound>
__global__ __launch_bounds__(kBound) void k_norm_backward(
    const uint16_t* dy, int64_t lddy, const void* x, int64_t n_rows, int d, int64_t ldx,
    const void* __restrict__ weight, int rms, const float* __restrict__ mean, const float* __restrict__ rstd, void* dx,
    int64_t lddx, float* __restrict__ parts) {
  backward_rows<kX, kW, kVecs, kBias>(dy, lddy, x, n_rows, d, ldx, weight, rms, mean, rstd, dx, lddx, parts,
                               static_cast<int>(gridDim.x));
}

// Column c of [count][ld] partial sums: 32 threads a column, each a fixed share of
// the rows in four sums, joined in order.
constexpr int kSumThreads = 1024;
constexpr int kSumCols = 32;
constexpr int kSumRows = kSumThreads / kSumCols;

__global__ __launch_bounds__(kSumThreads) void k_norm_sums(const float* __restrict__ parts, int count, int ld, int d,
                                                           float* __restrict__ dweight, float* __restrict__ dbias,
                                                           int accumulate) {
  __shared__ float s[kSumRows][kSumCols + 1];
  const int c = static_cast<int>(threadIdx.x) % kSumCols;
  const int k = static_cast<int>(threadIdx.x) / kSumCols;
  const int col = static_cast<int>(blockIdx.x) * kSumCols + c;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < ld) {
    const float* __restrict__ p = parts + col;
    int r = k;
    for (; r + 7 * kSumRows < count; r += 8 * kSumRows) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = p[static_cast<int64_t>(r + u * kSumRows) * ld];
#pragma unroll
      for (int u = 0; u < 8; ++u) a[u & 3] = a[u & 3] + x[u];
    }
    for (; r < count; r += kSumRows) a[0] = a[0] + p[static_cast<int64_t>(r) * ld];
  }
  s[k][c] = (a[0] + a[1]) + (a[2] + a[3]);
  __syncthreads();
#pragma unroll
  for (int o = kSumRows / 2; o >= 1; o >>= 1) {
    if (k < o) s[k][c] = s[k][c] + s[k + o][c];
    __syncthreads();
  }
  if (k == 0 && col < ld) {
    float* to = col < d ? dweight : dbias;
    const int at = col < d ? col : col - d;
    if (to) to[at] = accumulate ? to[at] + s[0][c] : s[0][c];
  }
}

// Few rows: a workgroup a row for dx, and beside them workgroups that each sum 64
// columns of dweight and dbias over all rows: one launch and no partial sums, for a
// second read of x and dy (so dx may not take their place here).
template <int kX, int kW, int kVecs, int kBound>
__global__ __launch_bounds__(kBound) void k_norm_backward_few(
    const uint16_t* __restrict__ dy, int64_t lddy, const void* __restrict__ x, int n_rows, int d, int64_t ldx,
    const void* __restrict__ weight, int rms, const float* __restrict__ mean, const float* __restrict__ rstd,
    void* __restrict__ dx, int64_t lddx, float* __restrict__ dweight, float* __restrict__ dbias, int accumulate,
    int row_blocks) {
  __shared__ float2 part[kMaxWaves][64];
  const int threads = static_cast<int>(blockDim.x);
  const int waves = threads >> 6;
  const int wave = static_cast<int>(threadIdx.x) >> 6;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    backward_rows<kX, kW, kVecs, false>(dy, lddy, x, n_rows, d, ldx, weight, rms, mean, rstd, dx, lddx, nullptr, row_blocks);
    return;
  }
  const int first = (static_cast<int>(blockIdx.x) - row_blocks) * 64;
  const int col = first + (lane & 7) * 8;  // 8 lanes a row
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
  if (col < d)
    for (int row = static_cast<int>(threadIdx.x) >> 3; row < n_rows; row += threads >> 3) {
      float f[8], g[8];
      widen<kX>(load8<kX>(x, row * ldx + col), f);
      widen<RLK_TYPE_BF16>(load8<RLK_TYPE_BF16>(dy, row * lddy + col), g);
      const float r = rstd[row];
      const float m = rms ? 0.0f : mean[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] = dw[e] + weight_term(g[e], (f[e] - m) * r);
        db[e] = db[e] + g[e];
      }
    }
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int o = 8; o <= 32; o *= 2) {
      dw[e] = dw[e] + __shfl_xor(dw[e], o);
      db[e] = db[e] + __shfl_xor(db[e], o);
    }
  if (lane < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[wave][lane * 8 + e] = make_float2(dw[e], db[e]);
  }
  __syncthreads();
  const int at = first + lane;
  if (wave == 0 && at < d) {
    float2 s = part[0][lane];
    for (int k = 1; k < waves; ++k) {
      s.x = s.x + part[k][lane].x;
      s.y = s.y + part[k][lane].y;
    }
    if (dweight) dweight[at] = accumulate ? dweight[at] + s.x : s.x;
    if (dbias) dbias[at] = accumulate ? dbias[at] + s.y : s.y;
  }
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static int32_t launched() { return hipGetLastError() == hipSuccess ? RLK_OK : RLK_ERR_HIP; }

static bool sizes_ok(int64_t n_rows, int64_t d) {
  return n_rows >= 0 && n_rows <= kMaxRows && d >= 8 && d <= kMaxD && d % 8 == 0;
}
static bool stride_ok(int64_t ld, int64_t d) { return ld >= d && ld % 8 == 0 && ld <= kMaxLd; }

// 8-value vectors a thread: 2, and 4 where a row needs more than 512 threads of 2.
static int vecs_for(int64_t d) { return d <= 16 * kMaxThreads ? 2 : 4; }
static int threads_for(int64_t d) {
  const int64_t a_wave = vecs_for(d) * 64;
  return static_cast<int>((d / 8 + a_wave - 1) / a_wave) * 64;
}

// Workgroups of a walk over the rows: `resident` threads a compute unit, all with
// the same number of rows but the last.
static int grid_for(int64_t n_rows, int64_t d, int resident) {
  const int64_t fit = resident / threads_for(d);
  const int64_t most = static_cast<int64_t>(kUnits) * (fit > 0 ? fit : 1);
  const int64_t rows = (n_rows + most - 1) / most;
  return rows > 0 ? static_cast<int>((n_rows + rows - 1) / rows) : 0;
}

// Threads a compute unit that the forward walk is cut for. Fewer are resident: k_norm's
// 80 to 90 registers leave 6 or 5 waves a SIMD (1536 or 1280 threads), 142 to 156 beyond d =
// 8192 leave 3, so the last workgroups start when others end (4999 x 2080: 2500 workgroups, 2048
// resident, 12.2 us on the GPU for 42 MB; 8192 x 4096 in float32 31 us at 6.4 TB/s).
constexpr int kForwardThreads = 2048;

// Calls f with the types, the vectors a thread and the largest workgroup as
// constants (a bound of 1024 threads leaves 128 registers: spills, and 403 us
// instead of 285 for the backward of 32768 x 8192). The backward of float32 x beyond d =
// 8192 with both sums still spills 14 registers (float32 weight: 32): 8192 x 16384 372 us, without
// dbias, which spills nothing, 267.
template <typename F>
static void by_type(int x_type, int w_type, int64_t d, const F& f) {
  using B = std::integral_constant<int, RLK_TYPE_BF16>;
  using S = std::integral_constant<int, RLK_TYPE_F32>;
  const auto sized = [&](auto xt, auto wt) {
    if (threads_for(d) <= 256)
      f(xt, wt, std::integral_constant<int, 2>(), std::integral_constant<int, 256>());
    else if (vecs_for(d) == 2)
      f(xt, wt, std::integral_constant<int, 2>(), std::integral_constant<int, kMaxThreads>());
    else
      f(xt, wt, std::integral_constant<int, 4>(), std::integral_constant<int, kMaxThreads>());
  };
  const auto typed = [&](auto xt) {
    if (w_type == RLK_TYPE_BF16)
      sized(xt, B());
    else
      sized(xt, S());
  };
  if (x_type == RLK_TYPE_BF16)
    typed(B());
  else
    typed(S());
}

// Resident threads a compute unit in the backward walk: 512 for large batches (65536
// x 4096 281 us, with 768 326; 16384 x 4096 82 and 86), 768 for others (65536 x 512 54
// us, with 512 61; 8192 x 4096 46 and 47).
constexpr int kBackwardThreads = 768;
constexpr int kBackwardThreadsLarge = 512;
constexpr int64_t kLarge = int64_t(1) << 25;  // values
static int backward_grid(int64_t n_rows, int64_t d) {
  return grid_for(n_rows, d, n_rows * d > kLarge ? kBackwardThreadsLarge : kBackwardThreads);
}
// Rows up to which dweight's columns are summed beside the rows in one launch (a
// call of 37 x 1000 15.0 us, in two launches 17.2; of 128 x 8192 14.9 and 17.1).
constexpr int kFewRows = 128;

}  // namespace rlk_norm_layer

extern "C" {

int32_t rlk_layer_norm(const void* x, int32_t x_type, int64_t n_rows, int64_t d, int64_t x_stride,
                       const void* weight, const void* bias, int32_t weight_type, int32_t kind, float eps,
                       uint16_t* y, int64_t y_stride, float* mean_out, float* rstd_out, hipStream_t stream) {
  using namespace rlk_norm_layer;
  if (!sizes_ok(n_rows, d) || !stride_ok(x_stride, d) || !stride_ok(y_stride, d)) return RLK_ERR_SHAPE;
  if ((x_type != RLK_TYPE_BF16 && x_type != RLK_TYPE_F32) ||
      (weight_type != RLK_TYPE_BF16 && weight_type != RLK_TYPE_F32) ||
      (kind != RLK_NORM_LAYER && kind != RLK_NORM_RMS) || !(eps >= 0.0f && eps <= 3.0e38f))
    return RLK_ERR_SHAPE;
  if (n_rows == 0) return RLK_OK;
  if (!x || !weight || !y) return RLK_ERR_NULL;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(y, 16) || !aligned(mean_out, 4) ||
      !aligned(rstd_out, 4))
    return RLK_ERR_ALIGN;
  if (y == x && (x_type != RLK_TYPE_BF16 || x_stride != y_stride)) return RLK_ERR_SHAPE;  // rows would meet other rows
  const dim3 grid(grid_for(n_rows, d, kForwardThreads)), block(threads_for(d));
  by_type(x_type, weight_type, d, [&](auto xt, auto wt, auto vecs, auto bound) {
    k_norm<xt, wt, vecs, bound><<<grid, block, 0, stream>>>(x, n_rows, static_cast<int>(d), x_stride, weight, bias,
                                                      kind == RLK_NORM_RMS, eps, y, y_stride, mean_out, rstd_out);
  });
  return launched();
}

size_t rlk_layer_norm_backward_workspace_bytes(int64_t n_rows, int64_t d) {
  using namespace rlk_norm_layer;
  if (!sizes_ok(n_rows, d)) return 0;
  const int64_t fit = kBackwardThreads / threads_for(d);
  const int64_t most = static_cast<int64_t>(kUnits) * (fit > 0 ? fit : 1);
  return static_cast<size_t>(n_rows < most ? n_rows : most) * static_cast<size_t>(d) * 8 + 16;
}

int32_t rlk_layer_norm_backward(const uint16_t* dy, int64_t dy_stride, const void* x, int32_t x_type,
                                int64_t n_rows, int64_t d, int64_t x_stride, const void* weight,
                                int32_t weight_type, int32_t kind, const float* mean, const float* rstd,
                                void* dx, int64_t dx_stride, float* dweight, float* dbias, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace rlk_norm_layer;
  if (!sizes_ok(n_rows, d) || !stride_ok(x_stride, d) || !stride_ok(dy_stride, d)) return RLK_ERR_SHAPE;
  if ((x_type != RLK_TYPE_BF16 && x_type != RLK_TYPE_F32) ||
      (weight_type != RLK_TYPE_BF16 && weight_type != RLK_TYPE_F32) ||
      (kind != RLK_NORM_LAYER && kind != RLK_NORM_RMS) || (accumulate != 0 && accumulate != 1))
    return RLK_ERR_SHAPE;
  if (dx && !stride_ok(dx_stride, d)) return RLK_ERR_SHAPE;
  if (!dx && !dweight && !dbias) return RLK_ERR_NULL;
  const int rms = kind == RLK_NORM_RMS;
  const bool sums = dweight || dbias;
  if (n_rows > 0 && (!dy || !x || !weight || !rstd || (!rms && !mean))) return RLK_ERR_NULL;
  if (sums && !workspace) return RLK_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(dbias, 16) || (sums && !aligned(workspace, 16)))
    return RLK_ERR_ALIGN;
  if (sums && workspace_bytes < rlk_layer_norm_backward_workspace_bytes(n_rows, d)) return RLK_ERR_WORKSPACE;
  if (n_rows == 0 && (!sums || accumulate)) return RLK_OK;
  if (n_rows > 0 && dx &&
      ((dx == x && dx_stride != x_stride) || (dx == dy && (x_type != RLK_TYPE_BF16 || dx_stride != dy_stride))))
    return RLK_ERR_SHAPE;  // rows would meet other rows
  const int teams = backward_grid(n_rows, d);
  float* parts = sums ? static_cast<float*>(workspace) : nullptr;
  const int with_bias = dbias != nullptr;
  int32_t st;
  if (sums && n_rows > 0 && n_rows <= kFewRows && dx != x && dx != dy) {
    const int rows = dx ? static_cast<int>(n_rows) : 0;
    const dim3 grid(rows + static_cast<int>((d + 63) / 64)), block(threads_for(d));
    by_type(x_type, weight_type, d, [&](auto xt, auto wt, auto vecs, auto bound) {
      k_norm_backward_few<xt, wt, vecs, bound><<<grid, block, 0, stream>>>(
          dy, dy_stride, x, static_cast<int>(n_rows), static_cast<int>(d), x_stride, weight, rms, mean, rstd, dx,
          dx_stride, dweight, dbias, accumulate, rows);
    });
    return launched();
  }
  if (n_rows > 0) {
    const dim3 grid(teams), block(threads_for(d));
    by_type(x_type, weight_type, d, [&](auto xt, auto wt, auto vecs, auto bound) {
      const auto go = [&](auto with) {
        k_norm_backward<xt, wt, vecs, with, bound><<<grid, block, 0, stream>>>(
            dy, dy_stride, x, n_rows, static_cast<int>(d), x_stride, weight, rms, mean, rstd, dx, dx_stride, parts);
      };
      if (with_bias)
        go(std::true_type());
      else
        go(std::false_type());
    });
    if ((st = launched()) != RLK_OK) return st;
  }
  if (!sums) return RLK_OK;
  const int ld = static_cast<int>(d) * (with_bias ? 2 : 1);
  k_norm_sums<<<dim3((ld + kSumCols - 1) / kSumCols), dim3(kSumThreads), 0, stream>>>(
      parts, teams, ld, static_cast<int>(d), dweight, dbias, accumulate);
  return launched();
}

}  // extern "C"
