// sscan_delta_device.h -- device helpers shared by the gated delta rule's kernels.
//
// Matrix products run on v_mfma_f32_16x16x32_bf16 with float32 accumulators.  Its
// operands are bf16, so a float32 factor is cut into three bf16 terms that hold its
// 24 significand bits exactly (x = t0 + t1 + t2, each term 8 bits), and a product
// keeps the terms whose magnitude reaches 2^-24 of the leading one: three products
// against an exact bf16 factor, six against another float32 one.  The result is as
// exact as a float32 FMA chain at 3/8 of the float32 matrix instruction's cost.
//
// Lane layout of the instruction (lane = 16 * qd + i): A holds row i, contraction
// indices 8 qd .. 8 qd + 7; B holds column i and the same indices; the result holds
// column i and rows 4 qd .. 4 qd + 3.  A result becomes the B factor of the next
// product without leaving its lane when two result tiles p = 0, 1 of a group of 32
// rows are given the rows  32 s + 8 (i >> 2) + 4 p + (i & 3)  at tile row i: lane
// group qd then holds rows 32 s + 8 qd + 4 p + r, its own eight contraction indices.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace sscan {
namespace delta {

typedef __bf16 bf16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;      // tokens per chunk
constexpr int kTerms = 3;   // bf16 terms of a float32 factor
constexpr int kFrags = 6;   // non-zero 16 x 32 fragments of a lower (or upper) triangular 64 x 64 matrix
constexpr int kFragBytes = 1024;
// Per-token factors of a chunk, kC floats each (G the running sum of g, rk and rq the
// inverse norms of k and q): c = exp(G) rk, d = exp(G_C - G) rk, e = scale exp(G) rq,
// exp(G_C) (repeated); for the backward pass also beta, rk, rq.
constexpr int kVecFloats = 4 * kC;
constexpr int kVecFloatsBwd = 7 * kC;

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// N-term factor: N = 1 an exact bf16 value, N = 3 a float32 value.
template <int N>
struct Frag {
  bf16x8 t[N];
};

// Pairs are rounded together and widened again from the packed word (a shift and a
// mask): eleven instructions for the three terms of two values.
__device__ __forceinline__ Frag<3> split(f32x8 x) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  u32x4 w[3];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    f32x2 y = {x[2 * p], x[2 * p + 1]};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      uint32_t packed = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
      asm("" : "+v"(packed));  // keeps the widening below from becoming a second rounding
      w[n][p] = packed;
      if (n < 2) {
        y[0] -= __builtin_bit_cast(float, packed << 16);
        y[1] -= __builtin_bit_cast(float, packed & 0xffff0000u);
      }
    }
  }
  return Frag<3>{{__builtin_bit_cast(bf16x8, w[0]), __builtin_bit_cast(bf16x8, w[1]), __builtin_bit_cast(bf16x8, w[2])}};
}

__device__ __forceinline__ Frag<3> split(f32x4 lo, f32x4 hi) {
  return split(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// c + a b, dropping the products below 2^-24 of the leading one; the small products
// are added first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mul(const Frag<NA>& a, const Frag<NB>& b, f32x4 c) {
#pragma unroll
  for (int sum = 2; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (sum - i >= 0 && sum - i < NB) c = mfma(a.t[i], b.t[sum - i], c);
  return c;
}

// Token (or state row) of tile m, tile row i, in the chained order above.
__device__ __forceinline__ int chained(int m, int i) { return 32 * (m >> 1) + 8 * (i >> 2) + 4 * (m & 1) + (i & 3); }

// Index of the fragment (tile m, contraction step s) of an upper triangular matrix, or -1.
__device__ constexpr int upper_frag(int m, int s) { return m < 2 ? 2 * m + s : (s == 1 ? m + 2 : -1); }

__device__ __forceinline__ int lane_id() { return int(threadIdx.x) & 63; }
// In a scalar register, so that what depends on it branches without masks.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6); }

// This block's place in an order whose neighbours run on one XCD and share its L2 (blocks
// go to the eight XCDs in turn): each XCD takes a contiguous part of the grid.
__device__ __forceinline__ unsigned xcd_block() {
  const unsigned q = gridDim.x >> 3, r = gridDim.x & 7, x = blockIdx.x & 7;
  return x * q + (x < r ? x : r) + (blockIdx.x >> 3);
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  return float(x);
}

// Chunk rows are read and written through buffer descriptors whose size ends with the
// last row: an access past it (or at kOutside) reads 0 or is dropped, so tails cost no
// branches.  Offsets
// are bytes from the chunk's first row, in 32 bits (the callers' token strides are
// limited to kDeltaMaxStride elements).
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr int kOutside = int(0x80000000u);  // an offset beyond every buffer

// p and bytes are the same in all lanes (read from the first, so that the descriptor is
// held in scalar registers).
__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = uint32_t(__builtin_amdgcn_readfirstlane(int(at)));
  const uint64_t hi = uint32_t(__builtin_amdgcn_readfirstlane(int(at >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(hi << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(int(bytes)), 0x00020000);
}

// `rows` rows of `size` elements `stride` apart, from p.
template <typename T>
__device__ __forceinline__ Buffer rows_of(const T* p, int rows, int64_t stride, int size) {
  return buffer_of(p, rows > 0 ? uint32_t(((rows - 1) * stride + size) * int64_t(sizeof(T))) : 0u);
}

__device__ __forceinline__ void load1(Buffer b, int off, bf16* x) {
  *x = __builtin_bit_cast(bf16, __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0));
}
__device__ __forceinline__ void load1(Buffer b, int off, float* x) {
  *x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}
__device__ __forceinline__ void store1(Buffer b, int off, bf16 x) {
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, x), b, off, 0, 0);
}
__device__ __forceinline__ void store1(Buffer b, int off, float x) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), b, off, 0, 0);
}
__device__ __forceinline__ void load_wide(Buffer b, int off, bf16x8* x) {
  *x = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}
__device__ __forceinline__ void load_wide(Buffer b, int off, f32x8* x) {
  const auto lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
  const auto hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off + 16, 0, 0));
  *x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// x, computed here and not before: keeps the compiler from holding the sums of x and
// many constants in registers across a whole loop instead of adding them where used.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Eight consecutive elements at byte offset off, of which those at `left` and beyond
// read as 0 (wide: 16-byte accesses; left is then at most 0 or at least 8).
template <typename T, typename V8>
__device__ __forceinline__ void load8(Buffer b, int off, int left, bool wide, V8* x) {
  if (wide) {
    load_wide(b, left > 0 ? off : kOutside, x);
  } else {
    off = here(off);
    left = here(left);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      T y;
      load1(b, j < left ? off + j * int(sizeof(T)) : kOutside, &y);
      (*x)[j] = y;
    }
  }
}

template <typename T, typename V8>
__device__ __forceinline__ void store8(Buffer b, int off, int left, bool wide, V8 x) {
  if (wide) {
    typedef unsigned W __attribute__((ext_vector_type(sizeof(V8) / 4)));
    const W w = __builtin_bit_cast(W, x);
    off = left > 0 ? off : kOutside;
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, b, off, 0, 0);
    if constexpr (sizeof(V8) == 32)
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4], w[5], w[6], w[7]}, b, off + 16, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) store1(b, j < left ? off + j * int(sizeof(T)) : kOutside, T(x[j]));
  }
}

// A state's columns in the accumulator layout, from or to rows of `ld` floats: lane_at
// is the byte offset of the lane's row 8 qd and column, or kOutside.
template <int kTiles>
__device__ __forceinline__ void load_state(Buffer b, int lane_at, int ld, f32x4 (&S)[kTiles]) {
  lane_at = here(lane_at);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x;
      load1(b, lane_at + (32 * (m >> 1) + 4 * (m & 1) + r) * ld * 4, &x);
      S[m][r] = x;
    }
}

template <int kTiles>
__device__ __forceinline__ void store_state(Buffer b, int lane_at, int ld, const f32x4 (&S)[kTiles]) {
  lane_at = here(lane_at);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) store1(b, lane_at + (32 * (m >> 1) + 4 * (m & 1) + r) * ld * 4, S[m][r]);
}

__device__ __forceinline__ Frag<1> as_frag(bf16x8 x) { return Frag<1>{{x}}; }
__device__ __forceinline__ Frag<3> as_frag(f32x8 x) { return split(x); }

template <typename T>
struct Io;
template <>
struct Io<bf16> {
  static constexpr int kN = 1;  // bf16 terms of an input
  typedef bf16x8 V8;
};
template <>
struct Io<float> {
  static constexpr int kN = 3;
  typedef f32x8 V8;
};

// LDS tile of bf16 rows of KP elements, in units of eight (16 bytes).  A row's units are
// permuted by its index, so that both ways of reading the tile touch every bank once:
// sixteen chained rows at one unit (row_at), and four consecutive rows at four units
// (the transposing reads of col_frag).
template <int KP>
struct Tile {
  static constexpr int kElems = kC * KP;  // of one term

  __device__ static __forceinline__ int swizzle(int row) {
    return KP == 64 ? 4 * ((row >> 1) & 1) + ((row >> 3) & 3) : 4 * (row & 3) + ((row >> 3) & 3);
  }
  __device__ static __forceinline__ int unit_at(int row, int unit) { return row * KP + ((unit ^ swizzle(row)) << 3); }
  __device__ static __forceinline__ int at(int row, int dim) { return unit_at(row, dim >> 3) + (dim & 7); }
};

// Four rows of sixteen columns, transposed: lane i of each group of sixteen receives
// column i.  The caller passes row (i >> 2), columns 4 (i & 3) .. + 3 of the group.
__device__ __forceinline__ bf16x4 read_tr(const bf16* p) {
  const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(p));
  return __builtin_bit_cast(bf16x4, r);
}

// Fragment whose row i (or column i) is a column of rows `ld` elements apart, and whose
// eight contraction indices are eight consecutive rows: p is where columns
// 4 (i & 3) .. + 3 of the sixteen start in row (i >> 2) of them.
__device__ __forceinline__ bf16x8 col_frag(const bf16* p, int ld) {
  const bf16x4 a = read_tr(p), b = read_tr(p + 4 * ld);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The same of a tile: rows r0 .. r0 + 7 (r0 a multiple of eight: their units are
// permuted alike), columns from col4.
template <int KP>
__device__ __forceinline__ bf16x8 col_frag(const bf16* tile, int r0, int col4) {
  const int row = r0 + ((lane_id() & 15) >> 2);
  return col_frag(tile + Tile<KP>::unit_at(row, col4 >> 3) + (col4 & 4), KP);
}

__device__ __forceinline__ bf16x8 row_frag(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }

// A sequence of J products whose fragments come from LDS through a ring of R sets: a
// set is read R - 1 products before it is used, since one read takes as long as several
// products.  load(j, set) reads, use(j, set) multiplies; the barrier keeps the compiler
// from moving LDS reads back to their uses.
template <int J, int R, typename Set, typename Load>
__device__ __forceinline__ void ring_start(Set (&ring)[R], Load load) {
#pragma unroll
  for (int j = 0; j < R - 1 && j < J; ++j) load(j, ring[j]);
  __builtin_amdgcn_sched_barrier(0x7f);
}

template <int J, int R, typename Set, typename Load, typename Use>
__device__ __forceinline__ void ring_run(Set (&ring)[R], Load load, Use use) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (j + R - 1 < J) load(j + R - 1, ring[(j + R - 1) % R]);
    __builtin_amdgcn_sched_barrier(0x7f);
    use(j, ring[j % R]);
  }
}

// The j-th non-zero fragment of a lower (upper) triangular matrix: tile and step.
__device__ constexpr int lower_m(int j) { return j < 2 ? j : (j + 2) >> 1; }
__device__ constexpr int lower_s(int j) { return j < 2 ? 0 : j & 1; }
__device__ constexpr int upper_m(int j) { return j < 4 ? j >> 1 : j - 2; }
__device__ constexpr int upper_s(int j) { return j < 4 ? j & 1 : 1; }

__device__ __forceinline__ int row_len(const int32_t* lengths, int64_t b, int64_t len) {
  // lengths outside 0..len are clamped; one value for the whole wave
  if (!lengths) return int(len);
  const int64_t n = lengths[b];
  return __builtin_amdgcn_readfirstlane(int(n < 0 ? 0 : (n > len ? len : n)));
}

// Decays below exp(-104) are zero in float32; the clamp keeps the running sums (and
// differences of them) finite for g = -inf, a reset of the state.  NaN passes.
__device__ __forceinline__ float clamp_decay(float g) { return g < -104.0f ? -104.0f : g; }

}  // namespace delta
}  // namespace sscan
