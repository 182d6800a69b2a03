// Verification of drafted tokens, and the C ABI declared in include/rlk_draft.h.
//
// Kernels:
//   k_draft<.., kWhole>  one workgroup a sequence (kWhole, many sequences) or
//                 several, each for a run of the row's pieces of 512 columns.
//                 Every wave finds where the sequence's accepted tokens end (64
//                 drafted tokens at a time: three numbers a token), then sums
//                 the weights of its pieces, max(p - q, 0) or p, in float64. A
//                 whole sequence is drawn from and written at once; else the
//                 sums go to the workspace and
//   k_draft_pick  a wave a sequence, finds the piece in which the running sum
//                 passes sample_u times the whole, reads that piece's columns
//                 again and writes the outputs.
// 1024 sequences x 3 drafted tokens of 151936 columns: 464 MB in 114 to 124 us
// (column by column, without the table of weights, 335 us). Vector issue takes 69
// us of it (92 instructions a piece of a row, 41.7M counted), LDS 45 us, 29 of
// them bank conflicts of the look-ups; the two overlap in part. 256 samples: 26
// us, a sequence's loads, table, sums and draw one after another. 1 x 4: 6 + 6
// us, dependent loads.
// Piece sums are formed in one order whichever kernel forms them, so a
// sequence's outputs do not depend on the batch.
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

constexpr int kPiece = kWave * 8;   // 512 columns: one 16-byte vector a lane
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxVocab = int64_t(1) << 30;

struct Args {
  rlk_scored_rows t;
  rlk_scored_rows d;      // logits NULL: point masses
  int64_t n_seq;
  int64_t n_draft;
  int64_t vocab_real;
  int n_pieces;
  const int64_t* start;
  const int64_t* token;
  const double* accept_u;
  const double* sample_u;
  int64_t* token_out;
  int32_t* accepted_out;
  float* policy_out;
  float* ref_out;
  double* sums;           // [n_seq][n_pieces]
};

// Where a sequence's accepted tokens end, and what is known of the rows there
// (uniform across the wave).
struct Stop {
  int64_t first;   // draft_start[s]
  int64_t count;   // drafted tokens
  int64_t k;       // accepted tokens
  int64_t token;   // the drafted token at k (k < count)
  bool in_range;   // draft_start is usable
  bool served;     // a token can be drawn at row k
  bool sampled;    // q has logits there (else, with k < count, a point mass)
  float t, lse, part, threshold;         // the target's row
  float logp;                            // its policy logprob of the drafted token
  float t_q, part_q, threshold_q;        // the draft's (sampled)
};

__device__ __forceinline__ bool unit(double u) { return u >= 0.0 && u < 1.0; }

// Whether a row has a policy: the forward call's status, a temperature that is
// one and, where the record's numbers count (greedy rows' lse_support is NaN),
// a finite sum and a threshold.
__device__ __forceinline__ bool usable(const rlk_support_state& st, float t) {
  return st.status >= 0 && rlk::temperature_valid(t) &&
         (t == 0.0f || (fabsf(st.lse_support) < INFINITY && st.threshold == st.threshold));
}

// One lane a place, the row behind the last drafted token included, so that all
// a wave needs comes in two rounds of loads (the offsets, the rest).
__device__ __forceinline__ Stop find_stop(const Args& a, int64_t s, int lane) {
  Stop r = {};
  r.first = a.start[s];
  const int64_t end = a.start[s + 1];
  r.count = end - r.first;
  r.in_range = r.first >= 0 && r.first <= end && end <= a.n_draft;
  if (!r.in_range) return r;
  const bool fair = unit(a.sample_u[s]);
  const bool drafter = a.d.logits != nullptr;
  for (int64_t k0 = 0; k0 <= r.count; k0 += kWave) {
    const int64_t k = k0 + lane < r.count ? k0 + lane : r.count;
    const int64_t i = r.first + k, row = i + s;
    const rlk_support_state st = a.t.support[row];
    const float t = a.t.temperature[row], lse = a.t.lse[row];
    rlk_support_state sq = {};
    float t_q = 0.0f, lp = 0.0f, lq = 0.0f;
    int64_t tok = 0;
    double u = 0.0;
    if (k < r.count) {
      tok = a.token[i];
      u = a.accept_u[i];
      lp = a.t.policy_logp[row];
      if (drafter) {
        t_q = a.d.temperature[i];
        lq = a.d.policy_logp[i];
        sq = a.d.support[i];
      }
    }
    const bool sampled = k < r.count && drafter && t_q != 0.0f;
    bool wrong = !usable(st, t), stays = false;
    if (k < r.count) {
      wrong |= lp != lp || tok < 0 || tok >= a.vocab_real || !unit(u) || (drafter && (!usable(sq, t_q) || lq != lq));
      if (!sampled) lq = 0.0f;  // a point mass
      // a drafted token of no policy mass is never accepted (also where the drafter gave it none)
      stays = !wrong && lp > -INFINITY && u < exp(static_cast<double>(lp) - static_cast<double>(lq));
    }
    const u64 stops = __ballot(!stays);
    if (stops == 0) continue;
    const int l = __builtin_amdgcn_readfirstlane(__ffsll(stops) - 1);
    const bool served = !wrong && fair;
    r.k = k0 + l;
    r.token = __shfl(tok, l, kWave);
    r.served = (__ballot(served) >> l) & 1;
    r.sampled = (__ballot(sampled) >> l) & 1;
    const auto from = [l](float v) {
      return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), l)));
    };
    r.t = from(t);
    r.lse = from(lse);
    r.part = from(st.lse_support);
    r.threshold = from(st.threshold);
    r.logp = from(lp);
    r.t_q = from(t_q);
    r.part_q = from(sq.lse_support);
    r.threshold_q = from(sq.threshold);
    break;
  }
  return r;
}

// e^y, to about 3 * 2^-53 of the value: y = n ln 2 + r with ln 2
// as its float64 and the rest of it (one fused step each), the series of e^r to r^12 (|r| <= ln(2) / 2 leaves 2e-16). n is
// rounded by an addition of 1.5 * 2^52, whose low word then holds it, and 2^n
// is added to the exponent (conversions and ldexp run at a quarter of the rate).
// Where the result nears the ends of the range ldexp takes over: 0 for y down to
// -inf, infinity for y up to +inf (n fits its word because y is held to +-1000).
// A drafter's weight (kDraft) stays finite, so that no p - q is a NaN and a sum
// with an infinite p is refused. y is a number: lse_support is finite, and a NaN
// logit never reaches the threshold.
template <bool kDraft>
__device__ __forceinline__ double exp_down(double y) {
  constexpr double kRound = 6755399441055744.0;
  const double c = fmin(fmax(y, -1000.0), kDraft ? 709.782712893384 : 1000.0);
  const double t = fma(c, 1.4426950408889634074, kRound);
  const double n = t - kRound;
  double r = fma(-n, 0x1.62e42fefa39efp-1, c);
  r = fma(-n, 0x1.abc9e3b39803fp-56, r);
  double p = 2.08767569878680989792e-09;  // 1 / 12!
  p = fma(p, r, 2.50521083854417187751e-08);
  p = fma(p, r, 2.75573192239858906526e-07);
  p = fma(p, r, 2.75573192239858906526e-06);
  p = fma(p, r, 2.48015873015873015873e-05);
  p = fma(p, r, 1.98412698412698412698e-04);
  p = fma(p, r, 1.38888888888888888889e-03);
  p = fma(p, r, 8.33333333333333333333e-03);
  p = fma(p, r, 4.16666666666666666667e-02);
  p = fma(p, r, 1.66666666666666666667e-01);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  const int e = static_cast<int>(static_cast<uint32_t>(__builtin_bit_cast(u64, t)));
  if (!(y > -700.0 && y < 700.0)) return ldexp(p, e);
  return __builtin_bit_cast(double, __builtin_bit_cast(u64, p) + (static_cast<u64>(static_cast<uint32_t>(e)) << 52));
}

// One side's policy over the columns of a row.
template <bool kDraft>
struct Policy {
  double inv_t;
  double part;      // lse_support
  float threshold;

  __device__ __forceinline__ Policy(float t, float lse_support, float thr)
      : inv_t(1.0 / static_cast<double>(t)), part(static_cast<double>(lse_support)), threshold(thr) {}

  // fl32(x / T): the float64 product with 1/T is within 2^-52 of the quotient.
  // x has 8 significant bits and T 24, so a quotient that is no midpoint of two
  // float32 values is at least 2^-49 away from one (and a 25-bit midpoint times
  // T never has 8 bits): rounding the product rounds the quotient. (Below the
  // normal range it may be one 2^-149 off, which no weight shows.)
  __device__ __forceinline__ float scaled(float x) const { return static_cast<float>(static_cast<double>(x) * inv_t); }

  __device__ __forceinline__ double mass(float x) const {
    return x >= threshold ? exp_down<kDraft>(static_cast<double>(scaled(x)) - part) : 0.0;
  }
};

// Weights by BF16 pattern: a row of 152,000 columns holds a few thousand
// distinct values, so a workgroup with many columns to weigh computes each
// once. The table covers magnitudes of 2^-12 to 64 of either sign, interleaved
// (slot 2 (m - kMagLo) + sign, m the 15-bit magnitude pattern); other values
// are computed where they stand.
constexpr uint32_t kMagLo = 0x3980u;                 // 2^-12
constexpr int kMags = 0x4280 - 0x3980;               // to 64: 18 binades of 128 values
constexpr int kSlots = 2 * kMags;                    // 36 KB of float64

__device__ __forceinline__ uint32_t slot_bits(int slot) {
  return (kMagLo + static_cast<uint32_t>(slot >> 1)) | (static_cast<uint32_t>(slot & 1) << 15);
}

// The slots of the two values of a word; at least kSlots where one is outside.
__device__ __forceinline__ uint32_t slots2(uint32_t w) {
  uint32_t sign, twice, slot;
  asm("v_pk_lshrrev_b16 %[sign], %[c15], %[w]\n\t"
      "v_pk_mad_u16 %[twice], %[w], %[c2], %[sign]\n\t"
      "v_pk_sub_u16 %[slot], %[twice], %[lo]"
      : [sign] "=&v"(sign), [twice] "=&v"(twice), [slot] "=&v"(slot)
      : [w] "v"(w), [c15] "v"(0x000F000Fu), [c2] "v"(0x00020002u), [lo] "v"(2u * kMagLo * 0x10001u));
  return slot;
}
static_assert(2u * kMagLo <= 0xFFFFu && kSlots <= 0xFFFF, "slots are 16-bit numbers");

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("v_pk_max_u16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Weights of the 8 columns of a vector, from the table where all 8 are in it.
template <bool kDraft>
__device__ __forceinline__ void look_up(const double* __restrict__ table, const Policy<kDraft>& p, const u32x4& v, double (&m)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = slots2(w[i]);
  const uint32_t top = pk_max(pk_max(s[0], s[1]), pk_max(s[2], s[3]));
  if ((top & 0xFFFFu) < kSlots && (top >> 16) < kSlots) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[2 * i] = table[s[i] & 0xFFFFu];
      m[2 * i + 1] = table[s[i] >> 16];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t slot = (s[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
      const uint32_t b = (w[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
      if (slot < kSlots)
        m[e] = table[slot];
      else
        m[e] = b == 0xFF80u ? 0.0 : p.mass(__uint_as_float(b << 16));
    }
  }
}

template <bool kDraft>
__device__ __forceinline__ void compute(const Policy<kDraft>& p, const u32x4& v, double (&m)[8]) {
  float x[8];
  rlk::unpack8(v, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) m[e] = p.mass(x[e]);
}

// What the columns of one sequence's row weigh.
struct Weights {
  const u32x4* p_row;
  const u32x4* q_row;    // NULL: no residual, or q is a point mass
  Policy<false> p;
  Policy<true> q;
  int64_t point;         // column of q's point mass, -1: none

  __device__ __forceinline__ Weights(const Args& a, int64_t s, const Stop& st)
      : p_row(reinterpret_cast<const u32x4*>(a.t.logits + (st.first + s + st.k) * a.t.row_stride)),
        q_row(st.sampled ? reinterpret_cast<const u32x4*>(a.d.logits + (st.first + st.k) * a.d.row_stride) : nullptr),
        p(st.t, st.part, st.threshold),
        q(st.t_q, st.part_q, st.threshold_q),
        point(st.k < st.count && !st.sampled ? st.token : -1) {}

  // Weights of a lane's 8 columns of a piece, given both sides' vectors and, with
  // kTable, tables. Columns from `real` on weigh nothing.
  template <bool kTable>
  __device__ __forceinline__ void columns(const u32x4& x, const u32x4& y, const double* __restrict__ table, int piece,
                                          int lane, int64_t real, double (&m)[8]) const {
    if constexpr (kTable)
      look_up(table, p, x, m);
    else
      compute(p, x, m);
    if (q_row != nullptr) {
      double n[8];
      if constexpr (kTable)
        look_up(table + kSlots, q, y, n);
      else
        compute(q, y, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = fmax(m[e] - n[e], 0.0);
    }
    const int64_t first = static_cast<int64_t>(piece) * kPiece;  // uniform, as both conditions are
    if (point >= first && point < first + kPiece) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (first + lane * 8 + e == point) m[e] = fmax(m[e] - 1.0, 0.0);
    }
    if (first + kPiece > real) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (first + lane * 8 + e >= real) m[e] = 0.0;
    }
  }
};

// Inclusive sums over the lanes, and the whole sum, on lane moves of the vector
// units (shuffles through LDS took most of a piece's time): within rows of 16
// lanes by 1, 2, 4 and 8, then row 0's total into row 1 and 2's into 3, then
// the lower half's into the upper.
template <int Ctrl, int RowMask>
__device__ __forceinline__ double moved(double v) {  // 0 where no lane is
  const u64 u = __builtin_bit_cast(u64, v);
  const uint32_t lo = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(static_cast<uint32_t>(u)), Ctrl, RowMask, 0xF, true));
  const uint32_t hi = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(static_cast<uint32_t>(u >> 32)), Ctrl, RowMask, 0xF, true));
  return __builtin_bit_cast(double, (static_cast<u64>(hi) << 32) | lo);
}

__device__ __forceinline__ double wave_scan(double v) {
  v = v + moved<0x111, 0xF>(v);
  v = v + moved<0x112, 0xF>(v);
  v = v + moved<0x114, 0xF>(v);
  v = v + moved<0x118, 0xF>(v);
  v = v + moved<0x142, 0xA>(v);
  v = v + moved<0x143, 0xC>(v);
  return v;
}

__device__ __forceinline__ double lane_value(double v, int l) {  // l uniform
  const u64 u = __builtin_bit_cast(u64, v);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(u)), l));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(u >> 32)), l));
  return __builtin_bit_cast(double, (static_cast<u64>(hi) << 32) | lo);
}

__device__ __forceinline__ double wave_sum(double v) { return lane_value(wave_scan(v), kWave - 1); }

// Greedy rows: a wave's record is its maximum's order key (16 bits) over the
// complement of its column, so the largest record is the lowest column of the
// largest value. -0 counts as 0.
__device__ __forceinline__ u64 greedy_key(float x, int64_t column) {
  const uint32_t b = x == 0.0f ? 0u : __float_as_uint(x) >> 16;
  const uint32_t key = (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
  return (static_cast<u64>(key) << 32) | static_cast<u64>(0xFFFFFFFFu - static_cast<uint32_t>(column));
}

__device__ __forceinline__ u64 wave_top(u64 v) {
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(v, d, kWave);
    v = o > v ? o : v;
  }
  return v;
}

// A lane's vector of a piece; behind the row's last vector (or the last piece
// asked for) -inf, which weighs nothing.
__device__ __forceinline__ u32x4 vector_at(const u32x4* row, int piece, int to, int vecs, int lane) {
  const int v = piece * kWave + lane;
  return piece < to && v < vecs ? __builtin_nontemporal_load(row + v) : rlk::neg_inf_vec();
}

template <int kBatch>
struct Vectors {   // of the pieces that a wave weighs together
  u32x4 x[kBatch];
  u32x4 y[kBatch];

  __device__ __forceinline__ void load(const Weights& w, int piece, int stride, int to, int vecs, int lane) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      x[b] = vector_at(w.p_row, piece + b * stride, to, vecs, lane);
      if (w.q_row != nullptr) y[b] = vector_at(w.q_row, piece + b * stride, to, vecs, lane);
    }
  }
};

// The sums of the pieces [from, to) of a row, one wave a piece, into sums[piece].
// `waves` waves share them; the next pieces' vectors are on their way while a
// wave weighs its pieces (`now` holds the first ones).
template <bool kTable, int kBatch>
__device__ __forceinline__ void sum_pieces(const Args& a, const Weights& w, const double* __restrict__ table, int from,
                                           int to, int wave, int waves, int lane, Vectors<kBatch> now,
                                           double* __restrict__ sums) {
  const int vecs = static_cast<int>((a.vocab_real + 7) / 8);
  for (int piece = from + wave; piece < to; piece += kBatch * waves) {
    Vectors<kBatch> next;
    next.load(w, piece + kBatch * waves, waves, to, vecs, lane);
    double sum[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      double m[8];
      w.columns<kTable>(now.x[b], now.y[b], table, piece + b * waves, lane, a.vocab_real, m);
      sum[b] = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[b] = sum[b] + m[e];
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      sum[b] = wave_sum(sum[b]);
      if (lane == 0 && piece + b * waves < to) sums[piece + b * waves] = sum[b];
    }
    now = next;
  }
}

// A greedy row's pieces: the wave's record in its first piece's place, 0 in the others'.
template <int kBatch>
__device__ __forceinline__ void top_pieces(const Args& a, const Weights& w, int from, int to, int wave, int waves, int lane,
                                           Vectors<kBatch> now, double* __restrict__ sums) {
  const int vecs = static_cast<int>((a.vocab_real + 7) / 8);
  float top = -INFINITY;
  int64_t column = -1;
  for (int piece = from + wave; piece < to; piece += kBatch * waves) {
    Vectors<kBatch> next;
    next.load(w, piece + kBatch * waves, waves, to, vecs, lane);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t at = (static_cast<int64_t>(piece + b * waves) * kWave + lane) * 8;
      float x[8];
      rlk::unpack8(now.x[b], x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < a.vocab_real && (column < 0 || x[e] > top)) {  // columns rise: the first of equal values stays
          top = x[e];
          column = at + e;
        }
      if (lane == 0 && piece + b * waves < to) sums[piece + b * waves] = 0.0;
    }
    now = next;
  }
  const u64 best = wave_top(column < 0 ? 0 : greedy_key(top, column));
  if (lane == 0 && from + wave < to) sums[from + wave] = __builtin_bit_cast(double, best);
}

// Piece sums of a sequence, 64 a register, for a wave that draws from them: all
// loads at once, before anything else is known. Longer rows read them in place.
constexpr int kHeld = 8;

struct Sums {
  const double* at;
  int n;
  bool held;
  double v[kHeld];

  __device__ __forceinline__ Sums(const double* sums, int n_pieces, int lane)
      : at(sums), n(n_pieces), held(n_pieces <= kHeld * kWave) {
    if (!held) return;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) v[i] = i * kWave + lane < n ? at[i * kWave + lane] : 0.0;
  }

  // f(register or load, first piece) over the 64-piece groups until it returns true
  template <typename F>
  __device__ __forceinline__ void each(int lane, F f) const {
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i * kWave < n && f(v[i], i * kWave)) return;
    } else {
      for (int c0 = 0; c0 < n; c0 += kWave)
        if (f(c0 + lane < n ? at[c0 + lane] : 0.0, c0)) return;
    }
  }
};

// Draws a token from the pieces' sums (one wave) and writes a sequence's outputs.
__device__ __forceinline__ void draw_and_write(const Args& a, int64_t s, const Stop& st, const Sums& sums, int lane) {
  const int64_t base = st.first + s;
  const int64_t row = base + st.k;
  int64_t pick = -1;
  float policy = NAN, ref = NAN;
  if (st.served) {
    if (st.t == 0.0f) {
      u64 best = 0;
      sums.each(lane, [&](double v, int) {
        const u64 o = __builtin_bit_cast(u64, v);
        best = o > best ? o : best;
        return false;
      });
      best = wave_top(best);
      pick = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      policy = 0.0f;
      ref = 0.0f;
    } else {
      double total = 0.0;
      sums.each(lane, [&](double v, int) {
        total = total + wave_sum(v);
        return false;
      });
      if (total > 0.0 && total < INFINITY) {
        const double want = a.sample_u[s] * total;
        // the first piece whose running sum passes `want`; by rounding none may: then the last with any weight
        double before = 0.0, at_before = 0.0;
        int piece = 0;
        sums.each(lane, [&](double v, int c0) {
          const double incl = before + wave_scan(v);
          const u64 over = __ballot(incl > want && v > 0.0);
          const u64 any = __ballot(v > 0.0);
          const int l = __builtin_amdgcn_readfirstlane(over != 0 ? __ffsll(over) - 1 : (any != 0 ? 63 - __clzll(any) : -1));
          if (l >= 0) {
            piece = c0 + l;
            at_before = lane_value(incl, l) - lane_value(v, l);
          }
          before = lane_value(incl, kWave - 1);
          return over != 0;
        });
        // its columns: the first whose running sum passes, else the last with any weight
        const Weights w(a, s, st);
        const int vecs = static_cast<int>((a.vocab_real + 7) / 8), v = piece * kWave + lane;
        const u32x4 x = v < vecs ? w.p_row[v] : rlk::neg_inf_vec();
        const u32x4 y = w.q_row != nullptr && v < vecs ? w.q_row[v] : rlk::neg_inf_vec();
        double m[8];
        w.columns<false>(x, y, nullptr, piece, lane, a.vocab_real, m);
        double mine = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine = mine + m[e];
        double c = at_before + (wave_scan(mine) - mine);
        int hit = -1, tail = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          c = c + m[e];
          if (m[e] > 0.0) {
            tail = e;
            if (hit < 0 && c > want) hit = e;
          }
        }
        const u64 hits = __ballot(hit >= 0), tails = __ballot(tail >= 0);
        const int l = hits != 0 ? __ffsll(hits) - 1 : (tails != 0 ? 63 - __clzll(tails) : -1);
        if (l >= 0) {
          const int mine_e = hits != 0 ? hit : tail;
          float x8[8], xt = 0.0f;
          rlk::unpack8(x, x8);
#pragma unroll
          for (int e = 0; e < 8; ++e) xt = e == mine_e ? x8[e] : xt;
          pick = (static_cast<int64_t>(piece) * kWave + l) * 8 + __shfl(mine_e, l, kWave);
          const double z = static_cast<double>(w.p.scaled(__shfl(xt, l, kWave)));
          policy = static_cast<float>(z - w.p.part);
          ref = static_cast<float>(z - static_cast<double>(st.lse));
        }
      } else if (total == 0.0 && st.k < st.count && st.logp > -INFINITY) {
        // p is nowhere above q: the drafted token
        pick = st.token;
        policy = st.logp;
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

constexpr int kWholePieces = 512;   // piece sums that stay in LDS

// The pieces' sums of a sequence, in `parts` workgroups; with kWhole (parts 1)
// in LDS, and the rest of its work. kTable: weights by table.
template <bool kTable, bool kWhole, int kN, int kBatch, int kWavesEach>
__global__ __launch_bounds__(kN, kWavesEach) void k_draft(Args a, int parts, int pieces_each) {
  __shared__ double table[kTable ? 2 * kSlots : 1];        // 72 KB: two workgroups a compute unit
  __shared__ double piece_sums[kWhole ? kWholePieces : 1];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int64_t s = blockIdx.x / static_cast<unsigned>(parts);
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(parts));
  const Stop st = find_stop(a, s, lane);
  double* sums = kWhole ? piece_sums : a.sums + s * a.n_pieces;
  if (st.in_range && st.served) {  // uniform across the workgroup
    const Weights w(a, s, st);
    const int from = part * pieces_each;
    const int to = from + pieces_each < a.n_pieces ? from + pieces_each : a.n_pieces;
    Vectors<kBatch> now;
    now.load(w, from + wave, kN / kWave, to, static_cast<int>((a.vocab_real + 7) / 8), lane);
    if (st.t == 0.0f) {
      top_pieces<kBatch>(a, w, from, to, wave, kN / kWave, lane, now, sums);
    } else {
      if (kTable) {
        for (int i = threadIdx.x; i < kSlots; i += kN) {
          const float x = __uint_as_float(slot_bits(i) << 16);
          table[i] = w.p.mass(x);
          if (w.q_row != nullptr) table[kSlots + i] = w.q.mass(x);
        }
        __syncthreads();
      }
      sum_pieces<kTable, kBatch>(a, w, table, from, to, wave, kN / kWave, lane, now, sums);
    }
  }
  if constexpr (kWhole) {
    __syncthreads();
    if (wave != 0) return;
    if (st.in_range)
      draw_and_write(a, s, st, Sums(sums, a.n_pieces, lane), lane);
    else if (lane == 0)
      a.accepted_out[s] = -1;
  }
}

__global__ __launch_bounds__(kWave) void k_draft_pick(Args a) {
  const int64_t s = blockIdx.x;
  const Sums sums(a.sums + s * a.n_pieces, a.n_pieces, threadIdx.x);
  const Stop st = find_stop(a, s, threadIdx.x);
  if (st.in_range)
    draw_and_write(a, s, st, sums, threadIdx.x);
  else if (threadIdx.x == 0)
    a.accepted_out[s] = -1;
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

static int64_t pieces(const rlk_vocab_layout* L) { return (L->vocab_real + kPiece - 1) / kPiece; }

// A table costs a wave of 16 about as much as weighing half a piece of both
// sides column by column, so it pays from one piece a wave on. From 129
// sequences on there is a compute unit for at most one each: the sequence is
// drawn from where it was summed (no second launch). Above 256, two workgroups
// of half the threads share a compute unit, so that one weighs while the other
// waits for its first rows or draws (1024 x 3: 117 us, with one of 1024 threads 126).
static int32_t launch(const Args& a, hipStream_t stream) {
  constexpr int kUnits = 256;
  if (a.n_seq > kUnits / 2 && a.n_pieces <= kWholePieces) {
    const dim3 grid(static_cast<unsigned>(a.n_seq));
    if (a.n_seq <= kUnits)
      k_draft<true, true, 1024, 2, 4><<<grid, dim3(1024), 0, stream>>>(a, 1, a.n_pieces);
    else
      k_draft<true, true, 512, 2, 4><<<grid, dim3(512), 0, stream>>>(a, 1, a.n_pieces);
    return launched();
  }
  const bool table = a.n_seq * a.n_pieces >= kUnits * 16;
  const int64_t wanted = table ? kUnits : 2 * kUnits;             // workgroups: one of 1024 or two of 512 threads
  const int64_t least = table ? 16 : 8;                           // pieces each: one a wave
  int64_t parts = wanted / a.n_seq > 1 ? wanted / a.n_seq : 1;
  int64_t each = (a.n_pieces + parts - 1) / parts;
  each = each > least ? each : least;
  parts = (a.n_pieces + each - 1) / each;
  const dim3 grid(static_cast<unsigned>(a.n_seq * parts));        // at most 2^22: more than `wanted` only at one part
  if (table)
    k_draft<true, false, 1024, 2, 4><<<grid, dim3(1024), 0, stream>>>(a, static_cast<int>(parts), static_cast<int>(each));
  else
    k_draft<false, false, 512, 1, 4><<<grid, dim3(512), 0, stream>>>(a, static_cast<int>(parts), static_cast<int>(each));
  const int32_t st = launched();
  if (st != RLK_OK) return st;
  k_draft_pick<<<dim3(static_cast<unsigned>(a.n_seq)), dim3(kWave), 0, stream>>>(a);
  return launched();
}

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
  return static_cast<size_t>(n_seq) * static_cast<size_t>(pieces(layout)) * sizeof(double);
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
  a.n_pieces = static_cast<int>(pieces(layout));  // at most 2^21
  a.start = draft_start;
  a.token = draft_token;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.token_out = token_out;
  a.accepted_out = accepted_out;
  a.policy_out = policy_out;
  a.ref_out = ref_out;
  a.sums = static_cast<double*>(workspace);
  return launch(a, stream);
}

}  // extern "C"
