// Tiles of a BF16 product on the matrix cores, operands in either memory order.
//
//   out[m][n] = sum_k A[m][k] * B[n][k],  A = a[m * lda + k] (K contiguous) or
//   a[k * lda + m] (K across rows); the same for B.
//
// A workgroup of 4 waves takes a tile of BM x BN; a wave's part is cut into 16 x
// 16 blocks of v_mfma_f32_16x16x32_bf16. K runs in slices of 32, one matrix
// instruction deep, through a ring of LDS buffers; panels go from global memory
// straight into LDS. Large products are bound by power here: bare 16x16x32
// instructions on random values run at 2.06 PFLOP/s on all compute units,
// 32x32x16, which move the accumulators twice as often, at 1.81.
//
// Operand with K contiguous: a slice is BM rows of 32 values (64 bytes), the
// four 16-byte chunks of row r permuted by an XOR; one ds_read_b128 gives a lane
// its 8 values.
//
// Operand with K across rows: a slice is 32 rows (k) of BM values, read with
// ds_read_b64_tr_b16: 16 lanes take a 4 (k) x 16 block, and lane t receives
// column t's 4 values; two of them are a lane's 8. The rows that are read together
// lie in the same banks, so the chunks of row k are permuted by an XOR with a
// function of k: the 32 lanes that read together cover all 64 banks once.
//
// Pipeline, in slices: while slice s is multiplied, the fragments of s + 1 are
// read into registers and the loads of s + kRing are issued, spread over the
// slice, into the buffer that s came from (its fragments were read in s - 1, and
// a barrier has passed). The barrier at the end of a slice waits until s + 2 has
// landed and leaves the younger loads in flight, so a load has (kRing - 2) slices
// to come. The ring runs on from tile to tile, over several short ones.
//
// Order of a sum: increasing k, the accumulator carried from instruction to
// instruction, whatever the tile's shape. 16x16x32 gives the bits of two
// 32x32x16 in a row, so the sums are bit for bit those of rlk_linear.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "bf16_store.hpp"
#include "logp_device.hpp"

namespace rlk_tiles {

constexpr int kThreads = 256;
constexpr int kSlice = 32;              // K of a slice: one matrix instruction deep
constexpr int kXcds = 8;
// Tiles of an XCD's 32 compute units: 4 x 8, so that its L2 serves each panel
// to several of them (as in rlk_linear).
constexpr int kGM = 4;
constexpr int kGN = 8;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* LdsPtr;
typedef __attribute__((address_space(3))) s16x4* LdsTr;
typedef __attribute__((address_space(3))) const bf16x8* LdsFrag;

constexpr int kRsrcWord3 = 0x00020000;  // gfx9 raw buffer: 32-bit data format, no swizzle

// f(0), f(1) .. f(n - 1) with constants, written out.
template <typename F, int... kI>
__device__ __forceinline__ void each(const F& f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>()), ...);
}

// The n below `count` whose turn first + n * span / count is t, or -1.
constexpr int at_slot(int t, int count, int first, int span) {
  for (int n = 0; n < count; ++n)
    if (first + n * span / count == t) return n;
  return -1;
}

// Shape of a workgroup's tile: WM x WN waves; kRing LDS buffers of a slice; kPer
// workgroups a compute unit.
template <int BM_, int BN_, int WM_, int WN_, int kRing_, int kPer_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kRing = kRing_, kPer = kPer_;
  static constexpr int MB = BM / WM / 16, NB = BN / WN / 16;  // blocks of a wave
  static constexpr int kLoadsA = BM / 64, kLoadsB = BN / 64;  // 1 KB loads a wave and slice
  static constexpr int kLoads = kLoadsA + kLoadsB;
  static constexpr int kBytesA = BM * kSlice * 2, kBytes = (BM + BN) * kSlice * 2;  // of a buffer
  static constexpr int kLds = kRing * kBytes;
  static_assert(WM * WN * 64 == kThreads && BM % 64 == 0 && BN % 64 == 0, "four waves, whole loads");
  static_assert(NB % 2 == 0 && kLds * kPer <= 160 * 1024, "blocks are stored in pairs; the LDS of a compute unit");
  static_assert(kRing >= 3 && (kRing - 2) * kLoads < 64, "the wait counter has 6 bits");
};

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6); }

// Permutations of a row's 16-byte chunks. K contiguous, 4 chunks a row, 4 rows in
// the 256 bytes of the banks: a ds_read_b128 is served for lanes 0-3, 12-15 and
// 20-27 together (then 4-11, 16-19 and 28-31, and the same of the upper half), so
// with lane l at row l % 16, chunk l / 16, rows q = r / 4 of 0 and 3 meet rows of 1
// and 2 one chunk on; 0, 2, 3, 1 for q = 0 .. 3 keeps them apart (counted: none).
__device__ __forceinline__ int swz_rows(int r) {
  const int q = (r >> 2) & 3;
  return (((q ^ (q >> 1)) & 1) << 1) | (q >> 1);
}
// K across rows, kWidth values a row: rows 0-3 and 8-11 (the blocks of 32 lanes) at
// one 32-byte piece lie in different banks.
template <int kWidth>
__device__ __forceinline__ int swz_k(int k) {
  return (kWidth >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1)) + 2 * ((k >> 3) & 1);
}

// One operand of one tile: where its first slice begins and what may be read.
// K contiguous: lim = bytes from p to the end of the last row's K. K across rows:
// lim = bytes of a row from p on, k_end rows. Both are multiples of a chunk: the
// range check cuts whole words.
struct Panel {
  const uint16_t* p;
  int lim;
};

__device__ __forceinline__ Panel panel_rows(const uint16_t* p, int rows, int ld, int k) {
  return Panel{p, (rows > 0 && k > 0) ? ((rows - 1) * ld + k) * 2 : 0};
}

__device__ __forceinline__ Panel panel_cols(const uint16_t* p, int64_t cols, int most) {
  return Panel{p, cols > 0 ? static_cast<int>(cols < most ? cols : most) * 2 : 0};
}

// The slices of a panel one after another, as buffer resources whose range check
// returns zeros for rows past the operand's end, and for k past k_end.
template <bool kAcross>
struct Stream {
  const uint16_t* p;
  int rec;         // K contiguous: bytes left from p; across: of a whole slice
  int rest, tail;  // across: rows left, bytes of the last slice when it is not whole

  __device__ __forceinline__ void begin(const Panel& t, int ld, int k_end) {
    p = t.p;
    rec = kAcross ? (kSlice - 1) * ld * 2 + t.lim : (k_end > 0 ? t.lim : 0);
    rest = !kAcross || t.lim > 0 ? k_end : 0;
    tail = (k_end % kSlice - 1) * ld * 2 + t.lim;  // looked at only where a row is left
  }
  __device__ __forceinline__ void none() {
    rec = 0;
    rest = 0;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t now() const {
    const int n = kAcross ? (rest >= kSlice ? rec : (rest > 0 ? tail : 0)) : (rec > 0 ? rec : 0);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, __builtin_amdgcn_readfirstlane(n), kRsrcWord3);
  }
  __device__ __forceinline__ void advance(int ld) {
    if (kAcross) {
      p += static_cast<int64_t>(ld) * kSlice;
      rest -= kSlice;
    } else {
      p += kSlice;
      rec -= kSlice * 2;
    }
  }
};

// This lane's byte offsets into a slice for its wave's loads. Load i of wave w
// fills 1 KB of LDS in lane order, from 1 KB * (kLoads w + i) of the operand's part on.
template <int kLoads>
struct Offsets {
  int at[kLoads];
};

template <bool kAcross, int kWidth>
__device__ __forceinline__ Offsets<kWidth / 64> offsets_for(int ld) {
  constexpr int kLoads = kWidth / 64;
  const int l = static_cast<int>(threadIdx.x) & 63;
  const int w = static_cast<int>(threadIdx.x) >> 6;
  Offsets<kLoads> o;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    if (kAcross) {  // kWidth / 8 chunks a row
      constexpr int kChunks = kWidth / 8;
      const int k = (w * kLoads + i) * (64 / kChunks) + l / kChunks;
      o.at[i] = k * ld * 2 + ((l % kChunks) ^ swz_k<kWidth>(k)) * 16;
    } else {        // 16 rows of 4 chunks
      const int r = (w * kLoads + i) * 16 + (l >> 2);
      o.at[i] = r * ld * 2 + ((l & 3) ^ swz_rows(r)) * 16;
    }
    asm volatile("" : "+v"(o.at[i]));  // kept, not formed again for every load
  }
  return o;
}

__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, int off, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)(lds), 16, off, 0, 0, 0);
}

// LDS addresses of a wave's fragments in the buffer that is read next: lane l
// takes row or column 16 n + l % 16 of block n, k = 8 (l / 16) .. + 7. Where K is
// contiguous blocks lie 1 KB apart; where it runs across rows the chunk
// permutation makes an address for each block.
template <bool kAcross, int kBlocks>
struct FragAt {
  static constexpr int kCount = kAcross ? kBlocks : 1;
  uint32_t at[kCount];
};

template <bool kAcross, int kBlocks, int kWidth>
__device__ __forceinline__ FragAt<kAcross, kBlocks> frag_at(uint32_t base, int w) {
  const int lane = threadIdx.x & 63;
  FragAt<kAcross, kBlocks> f;
#pragma unroll
  for (int n = 0; n < f.kCount; ++n) {
    if (kAcross) {
      const int k = 8 * (lane >> 4) + ((lane >> 2) & 3);  // row that this lane's address names
      const int chunk = (w * kBlocks + n) * 2 + ((lane >> 1) & 1);
      f.at[n] = base + k * kWidth * 2 + (chunk ^ swz_k<kWidth>(k)) * 16 + (lane & 1) * 8;
    } else {
      const int r = w * kBlocks * 16 + (lane & 15);
      f.at[n] = base + r * kSlice * 2 + ((lane >> 4) ^ swz_rows(r)) * 16;
    }
    asm volatile("" : "+v"(f.at[n]));
  }
  return f;
}

template <bool kAcross, int kBlocks, int kWidth>
__device__ __forceinline__ bf16x8 read_frag(const FragAt<kAcross, kBlocks>& f, int n) {
  if constexpr (kAcross) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(static_cast<uintptr_t>(f.at[n])));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(static_cast<uintptr_t>(f.at[n] + 4 * kWidth * 2)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    return *(LdsFrag)(static_cast<uintptr_t>(f.at[0] + n * 16 * kSlice * 2));
  }
}

// One matrix instruction, the accumulator where it is. (Of the builtin the compiler
// makes forms with another destination, and moves accumulators in the loop.) The
// compiler does not know that this is one: what it needs is waited for by settle().
__device__ __forceinline__ void mma(f32x4& c, const bf16x8& b, const bf16x8& a) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// Between writes of the accumulators by ordinary instructions and mma (2 wait
// states), and between mma and their reads (11 for this instruction): 32. The
// accumulators pass through before and after, so that the one is done by then and
// the other does not begin.
template <int kM, int kN>
__device__ __forceinline__ void settle(f32x4 (&acc)[kM][kN]) {
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
    if (turn == 0) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  }
}

// An accumulator's values in ordinary registers, for good: copies that the compiler
// may merge with the accumulator end in moves around mma.
__device__ __forceinline__ f32x4 taken(const f32x4& c) {
  f32x4 v;
  asm("v_accvgpr_read_b32 %0, %1" : "=v"(v.x) : "a"(c.x));
  asm("v_accvgpr_read_b32 %0, %1" : "=v"(v.y) : "a"(c.y));
  asm("v_accvgpr_read_b32 %0, %1" : "=v"(v.z) : "a"(c.z));
  asm("v_accvgpr_read_b32 %0, %1" : "=v"(v.w) : "a"(c.w));
  return v;
}

// A tile's product: panels and the end of K.
struct TileIn {
  Panel a, b;
  int k_end;
};

__device__ __forceinline__ int slices_of(int k_end) {
  const int n = (k_end + 2 * kSlice - 1) / (2 * kSlice);
  return 2 * (n > 0 ? n : 1);  // an empty sum still goes through two slices, of zeros
}

// The pipeline of a workgroup: operands' strides, where loads and fragments lie,
// the ring's position, and the fragments in registers. The loads run kRing slices
// ahead of the sums, over as many tiles as that is; `next(t)` gives them the
// workgroup's next tile, or false.
template <class S, bool kTA, bool kTB, class Next>
struct Tiles {
  typedef f32x4 Acc[S::MB][S::NB];

  Next next;
  int left;       // slices of the loads' tile

  int lda, ldb;
  uint8_t* ring;
  int buf;        // byte offset of the buffer that the slice at hand came from
  Offsets<S::kLoadsA> oa;
  Offsets<S::kLoadsB> ob;
  Stream<kTA> sa;  // slices still to be loaded
  Stream<kTB> sb;
  FragAt<kTA, S::MB> pa;  // in the buffer of the next slice
  FragAt<kTB, S::NB> pb;
  bf16x8 fa[2][S::MB], fb[2][S::NB];  // of the slice at hand and of the next, in turn

  __device__ __forceinline__ Tiles(const Next& n, uint8_t* smem, int lda_, int ldb_)
      : next(n), lda(lda_), ldb(ldb_), ring(smem) {
    oa = offsets_for<kTA, S::BM>(lda);
    ob = offsets_for<kTB, S::BN>(ldb);
  }

  __device__ __forceinline__ void load_a(__amdgpu_buffer_rsrc_t r, uint8_t* to, int j) {
    load_to_lds(r, oa.at[j], to + (wave_id() * S::kLoadsA + j) * 1024);
  }
  __device__ __forceinline__ void load_b(__amdgpu_buffer_rsrc_t r, uint8_t* to, int j) {
    load_to_lds(r, ob.at[j], to + S::kBytesA + (wave_id() * S::kLoadsB + j) * 1024);
  }

  // The loads go on to the next tile.
  __device__ __forceinline__ void go_on() {
    TileIn t;
    if (next(t)) {
      sa.begin(t.a, lda, t.k_end);
      sb.begin(t.b, ldb, t.k_end);
      left = slices_of(t.k_end);
    } else {
      sa.none();
      sb.none();
      left = 1 << 30;
    }
  }

  // Fills the ring and reads the first slice's fragments.
  __device__ __forceinline__ void start() {
    left = 0;
#pragma unroll 1
    for (int q = 0; q < S::kRing; ++q) {  // (written out it is kilobytes of code, read for the first time)
      if (left == 0) go_on();  // uniform
      --left;
      const __amdgpu_buffer_rsrc_t ra = sa.now();
      const __amdgpu_buffer_rsrc_t rb = sb.now();
      sa.advance(lda);
      sb.advance(ldb);
#pragma unroll
      for (int j = 0; j < S::kLoadsA; ++j) load_a(ra, ring + q * S::kBytes, j);
#pragma unroll
      for (int j = 0; j < S::kLoadsB; ++j) load_b(rb, ring + q * S::kBytes, j);
    }
    if (left == 0) go_on();  // sums() finds at least a slice to load
    landed();
    buf = 0;
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LdsPtr)(ring)));
    pa = frag_at<kTA, S::MB, S::BM>(lds, wave_m());
    pb = frag_at<kTB, S::NB, S::BN>(lds + S::kBytesA, wave_n());
#pragma unroll
    for (int i = 0; i < S::MB; ++i) fa[0][i] = read_frag<kTA, S::MB, S::BM>(pa, i);
#pragma unroll
    for (int j = 0; j < S::NB; ++j) fb[0][j] = read_frag<kTB, S::NB, S::BN>(pb, j);
    // every wave has read its part before the first slice's loads go into that buffer
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int n = 0; n < kAddresses; ++n) turn(n, S::kBytes);
  }

  __device__ __forceinline__ static int wave_m() { return (threadIdx.x >> 6) % S::WM; }
  __device__ __forceinline__ static int wave_n() { return (threadIdx.x >> 6) / S::WM; }

  // Fragment address n (A's, then B's) goes to another buffer.
  static constexpr int kAddresses = FragAt<kTA, S::MB>::kCount + FragAt<kTB, S::NB>::kCount;
  __device__ __forceinline__ void turn(int n, int by) {
    if (n < pa.kCount)
      pa.at[n] += by;
    else
      pb.at[n - pa.kCount] += by;
  }

  // The wave's LDS reads, the loads of the slice after next, then the workgroup.
  __device__ __forceinline__ static void landed() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((S::kRing - 2) * S::kLoads) : "memory");
  }

  // One slice: its matrix instructions, with the fragments of the next slice read
  // (in the first three quarters, so that none is waited for at the barrier) and a
  // slice's loads issued between them, into the buffer `to`. sched_barrier keeps
  // each group of instructions where it is written; without restrict every
  // fragment read waits for all loads.
  template <int kHalf>
  __device__ __forceinline__ void slice(Acc& acc, uint8_t* __restrict__ to) {
    constexpr int kSlots = S::MB * S::NB, kReads = S::MB + S::NB, kLater = kSlots / 2;
    constexpr int kTurn = (kReads - 1) * (kSlots * 3 / 4) / kReads + 1;  // after the last read
    static_assert(kReads * 4 <= kSlots * 3 && S::kLoadsA < kLater && kLater >= 4 && S::kLoadsB <= kSlots - kLater, "one of each a slot");
    const __amdgpu_buffer_rsrc_t ra = sa.now();
    __amdgpu_buffer_rsrc_t rb;
    int by;
    each([&](auto slot) __attribute__((always_inline)) {
      constexpr int t = slot, i = t / S::NB, j = t % S::NB;
      mma(acc[i][j], fb[kHalf][j], fa[kHalf][i]);
      constexpr int read = at_slot(t, kReads, 0, kSlots * 3 / 4);
      if constexpr (read >= 0 && read < S::MB)
        fa[kHalf ^ 1][read] = read_frag<kTA, S::MB, S::BM>(pa, read);
      else if constexpr (read >= 0)
        fb[kHalf ^ 1][read - S::MB] = read_frag<kTB, S::NB, S::BN>(pb, read - S::MB);
      constexpr int la = at_slot(t, S::kLoadsA, 1, kLater - 1);
      if constexpr (la >= 0) load_a(ra, to, la);
      if constexpr (t == kLater - 2) sa.advance(lda);
      if constexpr (t == kLater - 1) rb = sb.now();
      constexpr int lb = at_slot(t, S::kLoadsB, kLater, kSlots - kLater);
      if constexpr (lb >= 0) load_b(rb, to, lb);
      if constexpr (t == kTurn) {
        // the buffer that was read becomes the one at hand
        buf = buf + S::kBytes == S::kLds ? 0 : buf + S::kBytes;
        by = buf + S::kBytes == S::kLds ? S::kBytes - S::kLds : S::kBytes;
      }
#pragma unroll
      for (int n = 0; n < kAddresses; ++n)
        if (kTurn + n * (kSlots - kTurn) / kAddresses == t) turn(n, by);
      if constexpr (t == kSlots - 1) sb.advance(ldb);
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, kSlots>());
    landed();
  }

  // The sums of the next tile, n_slices long, into acc. Element e of block (i, j) in
  // lane l is row 16 i + l % 16, column 16 j + 4 (l / 16) + e of the wave's part (B's
  // fragment is the first operand).
  __device__ __forceinline__ void sums(Acc& acc, int n_slices) {
#pragma unroll
    for (int i = 0; i < S::MB; ++i)
#pragma unroll
      for (int j = 0; j < S::NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    settle(acc);
    // Pairs of slices up to the end of the sums or of the loads' tile, without a
    // branch in between (one for each slice costs 3% of the large products); a ring
    // of odd length ends the loads' tile inside a pair.
    int s = 0;
    do {
      const int even = left & ~1;
      const int run = n_slices - s < even ? n_slices - s : even;
      if constexpr (S::kRing % 2) {
        for (int k = 0; k < run; k += 2) {
          slice<0>(acc, ring + buf);
          slice<1>(acc, ring + buf);
        }
      } else {
        int k = 0;
        do {  // at least once
          slice<0>(acc, ring + buf);
          slice<1>(acc, ring + buf);
          k += 2;
        } while (k < run);
      }
      s += run;
      left -= run;
      if (S::kRing % 2 && left == 1 && s < n_slices) {
        slice<0>(acc, ring + buf);
        go_on();
        slice<1>(acc, ring + buf);
        s += 2;
        --left;
      }
      if (left == 0) go_on();
    } while (s < n_slices);
    settle(acc);
  }
};

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

// First tile index of workgroup b of `grid` (a multiple of 8), which runs on XCD b %
// 8: the XCD's workgroups take neighbouring tiles.
__device__ __forceinline__ int first_tile(int grid) {
  const int b = static_cast<int>(blockIdx.x);
  return (b % kXcds) * (grid / kXcds) + b / kXcds;
}

}  // namespace rlk_tiles
