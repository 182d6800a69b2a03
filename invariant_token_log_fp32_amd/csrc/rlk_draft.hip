// Verification of drafted tokens, and the C ABI declared in include/rlk_draft.h.
//
// Kernels:
//   k_draft_sums  a wave per (sequence, chunk of 2048 columns): finds where the
//                 sequence's accepted tokens end (64 drafted tokens at a time,
//                 again in every wave: three numbers a token), then sums the
//                 weights of its columns, max(p - q, 0) or p, in float64.
//   k_draft_pick  a wave per sequence: the chunk in which the running sum
//                 passes sample_u times the whole, that chunk's columns again,
//                 the outputs.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "logp_device.hpp"
#include "rlk_draft.h"
#include "rlk_logp.h"

namespace rlk_draft {

using rlk::kWave;
using rlk::u32x4;

typedef unsigned long long u64;

constexpr int kChunkVecs = 4;                          // 16-byte vectors of a lane in a chunk
constexpr int kChunk = kChunkVecs * kWave * 8;         // 2048 columns
constexpr int kThreads = 256;
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxVocab = int64_t(1) << 30;

struct Args {
  rlk_scored_rows t;
  rlk_scored_rows d;      // logits NULL: point masses
  int64_t n_seq;
  int64_t n_draft;
  int64_t vocab_real;
  int64_t n_chunks;
  const int64_t* start;
  const int64_t* token;
  const double* accept_u;
  const double* sample_u;
  int64_t* token_out;
  int32_t* accepted_out;
  float* policy_out;
  float* ref_out;
  double* sums;           // [n_seq][n_chunks]
};

// Where a sequence's accepted tokens end (uniform across the wave).
struct Stop {
  int64_t first;   // draft_start[s]
  int64_t count;   // drafted tokens
  int64_t k;       // accepted tokens
  bool in_range;   // draft_start is usable
  bool served;     // a token can be drawn at row k
};

__device__ __forceinline__ bool unit(double u) { return u >= 0.0 && u < 1.0; }

__device__ __forceinline__ Stop find_stop(const Args& a, int64_t s, int lane) {
  Stop r;
  r.first = a.start[s];
  const int64_t end = a.start[s + 1];
  r.count = end - r.first;
  r.k = 0;
  r.in_range = r.first >= 0 && r.first <= end && end <= a.n_draft;
  r.served = false;
  if (!r.in_range) return r;
  bool bad = false;
  r.k = r.count;
  for (int64_t k0 = 0; k0 < r.count; k0 += kWave) {
    const int64_t k = k0 + lane;
    bool stays = true, wrong = false;
    if (k < r.count) {
      const int64_t i = r.first + k;
      const int64_t row = i + s;
      const int64_t tok = a.token[i];
      const double u = a.accept_u[i];
      const float lp = a.t.policy_logp[row];
      float lq = 0.0f;
      wrong = a.t.support[row].status < 0 || lp != lp || tok < 0 || tok >= a.vocab_real || !unit(u);
      if (a.d.logits != nullptr && a.d.temperature[i] != 0.0f) {
        lq = a.d.policy_logp[i];
        wrong |= a.d.support[i].status < 0 || lq != lq;
      }
      // a drafted token of no policy mass is never accepted (also where the drafter gave it none)
      stays = !wrong && lp > -INFINITY && u < exp(static_cast<double>(lp) - static_cast<double>(lq));
    }
    const u64 stops = __ballot(!stays);
    if (stops != 0) {
      const int l = __ffsll(stops) - 1;
      r.k = k0 + l;
      bad = (__ballot(wrong) >> l) & 1;
      break;
    }
  }
  const int64_t row = r.first + s + r.k;
  const float t = a.t.temperature[row];
  const float part = a.t.support[row].lse_support;
  r.served = !bad && a.t.support[row].status >= 0 && rlk::temperature_valid(t) && (t == 0.0f || part == part) &&
             unit(a.sample_u[s]);
  return r;
}

// One side's policy over the columns of a row.
struct Policy {
  double inv_t;
  double part;      // lse_support
  float threshold;

  __device__ __forceinline__ Policy() : inv_t(0.0), part(0.0), threshold(INFINITY) {}
  __device__ __forceinline__ Policy(float t, const rlk_support_state& st)
      : inv_t(1.0 / static_cast<double>(t)), part(static_cast<double>(st.lse_support)), threshold(st.threshold) {}

  // fl32(x / T): the float64 product with 1/T is within 2^-52 of the quotient.
  // x has 8 significant bits and T 24, so a quotient that is no midpoint of two
  // float32 values is at least 2^-49 away from one (and a 25-bit midpoint times
  // T never has 8 bits): rounding the product rounds the quotient. (Below the
  // normal range it may be one 2^-149 off, which no weight shows.)
  __device__ __forceinline__ float scaled(float x) const { return static_cast<float>(static_cast<double>(x) * inv_t); }

  __device__ __forceinline__ double mass(float x) const {
    return x >= threshold ? exp(static_cast<double>(scaled(x)) - part) : 0.0;
  }
};

// What the columns of one sequence's row weigh.
struct Weights {
  const u32x4* p_row;
  const u32x4* q_row;    // NULL: no residual, or q is a point mass
  Policy p;
  Policy q;
  int64_t point;         // column of q's point mass, -1: none

  __device__ __forceinline__ Weights(const Args& a, int64_t s, const Stop& st) {
    const int64_t row = st.first + s + st.k;
    p_row = reinterpret_cast<const u32x4*>(a.t.logits + row * a.t.row_stride);
    p = Policy(a.t.temperature[row], a.t.support[row]);
    q_row = nullptr;
    point = -1;
    if (st.k < st.count) {
      const int64_t i = st.first + st.k;
      if (a.d.logits != nullptr && a.d.temperature[i] != 0.0f) {
        q_row = reinterpret_cast<const u32x4*>(a.d.logits + i * a.d.row_stride);
        q = Policy(a.d.temperature[i], a.d.support[i]);
      } else {
        point = a.token[i];
      }
    }
  }

  // Weights of the 8 columns of vector v (columns from `real` on weigh nothing).
  __device__ __forceinline__ void columns(int64_t v, int64_t real, double (&w)[8]) const {
    float x[8], y[8];
    rlk::unpack8(p_row[v], x);
    if (q_row != nullptr) rlk::unpack8(q_row[v], y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = v * 8 + e;
      double m = c < real ? p.mass(x[e]) : 0.0;
      if (q_row != nullptr) m = c < real ? fmax(m - q.mass(y[e]), 0.0) : 0.0;
      if (c == point) m = fmax(m - 1.0, 0.0);
      w[e] = m;
    }
  }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1) v = v + __shfl_xor(v, d, kWave);
  return v;
}

// Greedy rows: a chunk's record is its maximum's order key (16 bits) over the
// complement of its column, so the largest record is the lowest column of the
// largest value. -0 counts as 0.
__device__ __forceinline__ u64 greedy_key(uint32_t b, int64_t column) {
  b = b == 0x8000u ? 0u : b;
  const uint32_t key = (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
  return (static_cast<u64>(key) << 32) | static_cast<u64>(0xFFFFFFFFu - static_cast<uint32_t>(column));
}

__global__ __launch_bounds__(kThreads) void k_draft_sums(Args a, int64_t n_work) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t work = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) + (threadIdx.x / kWave);
  if (work >= n_work) return;
  const int64_t s = work / a.n_chunks;
  const int64_t chunk = work % a.n_chunks;
  const Stop st = find_stop(a, s, lane);
  if (!st.in_range || !st.served) return;
  const Weights w(a, s, st);
  const int64_t v0 = chunk * (kChunk / 8);
  const bool greedy = a.t.temperature[st.first + s + st.k] == 0.0f;
  if (greedy) {
    u64 best = 0;
    for (int u = 0; u < kChunkVecs; ++u) {
      const int64_t v = v0 + u * kWave + lane;
      if (v * 8 >= a.vocab_real) break;
      const u32x4 x = w.p_row[v];
      const uint32_t bits[4] = {x.x, x.y, x.z, x.w};
      for (int e = 0; e < 8; ++e) {
        const int64_t c = v * 8 + e;
        const u64 key = greedy_key((bits[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu, c);
        if (c < a.vocab_real && key > best) best = key;
      }
    }
    for (int d = kWave / 2; d >= 1; d >>= 1) {
      const u64 o = __shfl_xor(best, d, kWave);
      best = o > best ? o : best;
    }
    if (lane == 0) a.sums[s * a.n_chunks + chunk] = __builtin_bit_cast(double, best);
    return;
  }
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < kChunkVecs; ++u) {
    const int64_t v = v0 + u * kWave + lane;
    if (v * 8 < a.vocab_real) {
      double m[8];
      w.columns(v, a.vocab_real, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = sum + m[e];
    }
  }
  sum = wave_sum(sum);
  if (lane == 0) a.sums[s * a.n_chunks + chunk] = sum;
}

__device__ __forceinline__ double wave_scan(double v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_up(v, d, kWave);
    if (lane >= d) v = v + o;
  }
  return v;
}

__global__ __launch_bounds__(kWave) void k_draft_pick(Args a) {
  const int lane = threadIdx.x;
  const int64_t s = blockIdx.x;
  const Stop st = find_stop(a, s, lane);
  if (!st.in_range) {
    if (lane == 0) a.accepted_out[s] = -1;
    return;
  }
  const int64_t base = st.first + s;
  const int64_t row = base + st.k;
  int64_t pick = -1;
  float policy = NAN, ref = NAN;
  if (st.served) {
    const float t = a.t.temperature[row];
    const double* sums = a.sums + s * a.n_chunks;
    const Weights w(a, s, st);
    if (t == 0.0f) {
      u64 best = 0;
      for (int64_t c = lane; c < a.n_chunks; c += kWave) {
        const u64 o = __builtin_bit_cast(u64, sums[c]);
        best = o > best ? o : best;
      }
      for (int d = kWave / 2; d >= 1; d >>= 1) {
        const u64 o = __shfl_xor(best, d, kWave);
        best = o > best ? o : best;
      }
      pick = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      policy = 0.0f;
      ref = 0.0f;
    } else {
      double total = 0.0;
      for (int64_t c0 = 0; c0 < a.n_chunks; c0 += kWave) {
        const double v = c0 + lane < a.n_chunks ? sums[c0 + lane] : 0.0;
        total = total + __shfl(wave_scan(v, lane), kWave - 1, kWave);
      }
      if (total > 0.0 && total < INFINITY) {
        const double want = a.sample_u[s] * total;
        // the first chunk whose running sum passes `want`; by rounding none may: then the last with any weight
        double before = 0.0, at_before = 0.0;
        int64_t chunk = -1;
        for (int64_t c0 = 0; c0 < a.n_chunks; c0 += kWave) {
          const double v = c0 + lane < a.n_chunks ? sums[c0 + lane] : 0.0;
          const double incl = before + wave_scan(v, lane);
          const u64 over = __ballot(incl > want && v > 0.0);
          const u64 any = __ballot(v > 0.0);
          const int l = over != 0 ? __ffsll(over) - 1 : (any != 0 ? 63 - __clzll(any) : -1);
          if (l >= 0) {
            chunk = c0 + l;
            at_before = __shfl(incl, l, kWave) - __shfl(v, l, kWave);
          }
          if (over != 0) break;
          before = __shfl(incl, kWave - 1, kWave);
        }
        // the columns of that chunk, 512 at a time
        double run = at_before;
        int64_t last = -1;
        bool found = false;
        for (int u = 0; u < kChunkVecs && !found; ++u) {
          const int64_t v = chunk * (kChunk / 8) + u * kWave + lane;
          double m[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
          if (v * 8 < a.vocab_real) w.columns(v, a.vocab_real, m);
          double mine = 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e) mine = mine + m[e];
          const double incl = wave_scan(mine, lane);
          double c = run + (incl - mine);
          int hit = -1, tail = -1;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c = c + m[e];
            if (m[e] > 0.0) {
              tail = e;
              if (hit < 0 && c > want) hit = e;
            }
          }
          const u64 hits = __ballot(hit >= 0);
          const u64 tails = __ballot(tail >= 0);
          if (hits != 0) {
            const int l = __ffsll(hits) - 1;
            last = (chunk * (kChunk / 8) + u * kWave + l) * 8 + __shfl(hit, l, kWave);
            found = true;
          } else if (tails != 0) {
            const int l = 63 - __clzll(tails);
            last = (chunk * (kChunk / 8) + u * kWave + l) * 8 + __shfl(tail, l, kWave);
          }
          run = run + __shfl(incl, kWave - 1, kWave);
        }
        pick = last;
        if (pick >= 0) {
          const float x = __uint_as_float(static_cast<uint32_t>(a.t.logits[row * a.t.row_stride + pick]) << 16);
          const double z = static_cast<double>(w.p.scaled(x));
          policy = static_cast<float>(z - w.p.part);
          ref = static_cast<float>(z - static_cast<double>(a.t.lse[row]));
        }
      } else if (total == 0.0 && st.k < st.count && a.t.policy_logp[row] > -INFINITY) {
        // p is nowhere above q: the drafted token
        pick = a.token[st.first + st.k];
        policy = a.t.policy_logp[row];
        ref = a.t.ref_logp[row];
      }
    }
  }
  for (int64_t k = lane; k <= st.count; k += kWave) {
    const bool kept = k < st.k, drawn = k == st.k;
    a.token_out[base + k] = kept ? a.token[st.first + k] : (drawn ? pick : -1);
    a.policy_out[base + k] = kept ? a.t.policy_logp[base + k] : (drawn ? policy : 0.0f);
    a.ref_out[base + k] = kept ? a.t.ref_logp[base + k] : (drawn ? ref : 0.0f);
  }
  if (lane == 0) a.accepted_out[s] = static_cast<int32_t>(st.k);
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static int32_t launched() { return hipGetLastError() == hipSuccess ? RLK_OK : RLK_ERR_HIP; }

static int32_t check_layout(const rlk_vocab_layout* L) {
  if (L == nullptr) return RLK_ERR_NULL;
  if (L->n_shards != 8) return RLK_ERR_SHAPE;
  if (L->vocab_padded < 64 || L->vocab_padded > kMaxVocab || L->vocab_padded % 64 != 0) return RLK_ERR_SHAPE;
  if (L->vocab_real < 1 || L->vocab_real > L->vocab_padded) return RLK_ERR_SHAPE;
  if (L->row_stride < L->vocab_padded || L->row_stride % 8 != 0) return RLK_ERR_SHAPE;
  if (!(L->groups == 1 || L->groups == 2 || L->groups == 4 || L->groups == 8)) return RLK_ERR_GROUPS;
  return RLK_OK;
}

static int64_t chunks(const rlk_vocab_layout* L) { return (L->vocab_real + kChunk - 1) / kChunk; }

static int32_t check_rows(const rlk_scored_rows* r, int64_t need, const rlk_vocab_layout* L) {
  if (r->n_rows < need || r->n_rows > 2 * kMaxRows) return RLK_ERR_SHAPE;
  if (r->row_stride < L->vocab_padded || r->row_stride % 8 != 0) return RLK_ERR_SHAPE;
  if (r->n_rows > 0 && r->row_stride > INT64_MAX / 2 / r->n_rows) return RLK_ERR_SHAPE;
  return RLK_OK;
}

}  // namespace rlk_draft

extern "C" {

size_t rlk_draft_workspace_bytes(int64_t n_seq, const rlk_vocab_layout* layout) {
  using namespace rlk_draft;
  if (check_layout(layout) != RLK_OK || n_seq < 0 || n_seq > kMaxRows) return 0;
  return static_cast<size_t>(n_seq) * static_cast<size_t>(chunks(layout)) * sizeof(double);
}

int32_t rlk_draft_verify(const rlk_scored_rows* target, const rlk_scored_rows* draft,
                         const rlk_vocab_layout* layout, int64_t n_seq, int64_t n_draft,
                         const int64_t* draft_start, const int64_t* draft_token, const double* accept_u,
                         const double* sample_u, int64_t* token_out, int32_t* accepted_out, float* policy_out,
                         float* ref_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace rlk_draft;
  int32_t st = check_layout(layout);
  if (st != RLK_OK) return st;
  if (target == nullptr) return RLK_ERR_NULL;
  if (n_seq < 0 || n_seq > kMaxRows || n_draft < 0 || n_draft > kMaxRows) return RLK_ERR_SHAPE;
  if ((st = check_rows(target, n_draft + n_seq, layout)) != RLK_OK) return st;
  if (draft != nullptr && (st = check_rows(draft, n_draft, layout)) != RLK_OK) return st;
  if (n_seq == 0) return RLK_OK;
  if (!target->logits || !target->temperature || !target->policy_logp || !target->ref_logp || !target->lse ||
      !target->support || !draft_start || !sample_u || !token_out || !accepted_out || !policy_out || !ref_out ||
      !workspace)
    return RLK_ERR_NULL;
  if (n_draft > 0 && (!draft_token || !accept_u)) return RLK_ERR_NULL;
  const bool drafted = draft != nullptr && n_draft > 0;
  if (drafted && (!draft->logits || !draft->temperature || !draft->policy_logp || !draft->support)) return RLK_ERR_NULL;
  if (!aligned(target->logits, 16) || !aligned(target->temperature, 4) || !aligned(target->policy_logp, 4) ||
      !aligned(target->ref_logp, 4) || !aligned(target->lse, 4) || !aligned(target->support, 4) ||
      !aligned(draft_start, 8) || !aligned(draft_token, 8) || !aligned(accept_u, 8) || !aligned(sample_u, 8) ||
      !aligned(token_out, 8) || !aligned(accepted_out, 4) || !aligned(policy_out, 4) || !aligned(ref_out, 4) ||
      !aligned(workspace, 16))
    return RLK_ERR_ALIGN;
  if (drafted && (!aligned(draft->logits, 16) || !aligned(draft->temperature, 4) || !aligned(draft->policy_logp, 4) ||
                  !aligned(draft->support, 4)))
    return RLK_ERR_ALIGN;
  if (workspace_bytes < rlk_draft_workspace_bytes(n_seq, layout)) return RLK_ERR_WORKSPACE;
  Args a;
  a.t = *target;
  a.d = drafted ? *draft : rlk_scored_rows{};
  a.n_seq = n_seq;
  a.n_draft = n_draft;
  a.vocab_real = layout->vocab_real;
  a.n_chunks = chunks(layout);
  a.start = draft_start;
  a.token = draft_token;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.token_out = token_out;
  a.accepted_out = accepted_out;
  a.policy_out = policy_out;
  a.ref_out = ref_out;
  a.sums = static_cast<double*>(workspace);
  const int64_t n_work = n_seq * a.n_chunks;
  const int64_t blocks = (n_work + kThreads / kWave - 1) / (kThreads / kWave);
  if (blocks > INT32_MAX) return RLK_ERR_SHAPE;
  k_draft_sums<<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream>>>(a, n_work);
  if ((st = launched()) != RLK_OK) return st;
  k_draft_pick<<<dim3(static_cast<unsigned>(n_seq)), dim3(kWave), 0, stream>>>(a);
  return launched();
}

}  // extern "C"
