// sscan_rec_tile.h -- how the recurrence's kernels cut a call into tiles, and how the tiles
// of a row hand the state on.
//
// A wave holds T tokens of 64 C consecutive channels, C of them a lane, and a block's waves
// hold consecutive tokens: a segment of a row.  A segment maps its entry state to its exit
// state by h -> A h + H, A the product of its decays and H its exit state from zero.  Where a
// row has several segments they run at once, and inputs are read once: a segment's block
// publishes its map as soon as it has one (the row's first: its exit state, as a map of
// nothing), joins the maps of the segments before it in its run of kRun segments, and applies
// them to the state that enters the run, which the last segment of the run before publishes.
// So a chain over the row has a link for each run only, and every state is computed in one
// order, whatever the order of arrival.  Only the first segment reads the row's entry state:
// the last one may write its exit state over it.
//
// The waits for other blocks have to end whatever the order in which blocks start: a block
// takes the number of its segment from a counter when it starts, the first segments of all
// rows first.  Those it waits for have lower numbers, so their blocks run already, and the
// lowest of them waits for nobody.
//
// Maps and states are words of 64 bits, written and read whole (no fence orders them against
// anything else): the upper half is A's bits, never kEmpty's, the lower half H's or the
// state's.  A small kernel empties them before.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sscan_rec_device.h"

namespace sscan {
namespace rec {

constexpr uint32_t kEmpty = 0xffffffffu;
// Segments of a run: fewer maps to join and more links of the chain.  Forward of 8 x 4096 x
// 4096 bf16: runs of 16 291 us, of 8 285, of 4 282; one row of 65536 x 1536: 225, 220, 238.
constexpr int kRun = 8;
constexpr int kMaxWaves = 16;        // of a block

struct TileArgs {
  RecArgs a;
  uint64_t* maps;                    // [nseg][batch][groups * 64 C]
  uint64_t* states;                  // [runs][batch][groups * 64 C]: the state that leaves a run
  unsigned* ticket;                  // segments handed out
  float* entry;                      // [ceil(len / entry_step)][batch][groups * 64 C]: the gradients' entry states
  int entry_step;
  int nseg;
  unsigned groups;                   // of 64 C channels
};

__device__ __forceinline__ void publish(uint64_t* at, uint32_t hi, float lo) {
  const uint64_t w = uint64_t(hi) << 32 | __float_as_uint(lo);
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint32_t map_bits(float a) {
  const uint32_t u = __float_as_uint(a);
  return u == kEmpty ? 0x7fc00000u : u;
}

// Reads n words `pitch` apart, C a lane, in order, as soon as they are there: f(c, A, H)
// of each.  All lanes of a wave go on together; four places (two, of four channels) are read
// at once.  A wait of 2^24 reads is many seconds long and cannot happen; it ends, with NaN,
// instead of never.
template <int C, typename F>
__device__ __forceinline__ void read_words(const uint64_t* at, int64_t pitch, int n, F f) {
  constexpr int kAhead = C == 4 ? 2 : 4;
  int done = 0;
  for (int tries = 0; done < n; ++tries) {
    uint64_t w[kAhead][C];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c)
        w[k][c] = __hip_atomic_load(at + (done + k < n ? done + k : n - 1) * pitch + c, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    const int first = done;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      bool ready = true;
#pragma unroll
      for (int c = 0; c < C; ++c) ready = ready && uint32_t(w[k][c] >> 32) != kEmpty;
      if (done == first + k && done < n && (!__ballot(!ready) || tries > (1 << 24))) {
#pragma unroll
        for (int c = 0; c < C; ++c) f(c, __uint_as_float(uint32_t(w[k][c] >> 32)), __uint_as_float(uint32_t(w[k][c])));
        ++done;
      }
    }
  }
}

// The state that enters segment `seg` > 0: the lane's words lie `pitch` apart from segment to
// segment (of the maps) and from run to run (of the states).
template <int C>
__device__ __forceinline__ void enter(const uint64_t* maps, const uint64_t* states, int64_t pitch, int seg, float (&h)[C]) {
  const int run = seg / kRun, inside = seg % kRun;
  float A[C], H[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = 1.0f;
    H[c] = 0.0f;
    h[c] = 0.0f;
  }
  read_words<C>(maps + int64_t(run) * kRun * pitch, pitch, inside, [&](int c, float a, float b) {
    A[c] *= a;
    H[c] = fmaf(a, H[c], b);
  });
  if (run > 0) read_words<C>(states + int64_t(run - 1) * pitch, pitch, 1, [&](int c, float, float b) { h[c] = b; });
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = fmaf(A[c], h[c], H[c]);
}

// Empties the words (n pairs of them) and sets the counters to 0.
__global__ __launch_bounds__(256) static void clear_kernel(uint4* words, int64_t n, unsigned* tickets) {
  for (int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x; k < n; k += int64_t(gridDim.x) * 256)
    words[k] = uint4{kEmpty, kEmpty, kEmpty, kEmpty};
  if (blockIdx.x == 0 && threadIdx.x < 2) tickets[threadIdx.x] = 0;
}

// C elements, and the same at any address that an element can have.
template <typename IO, int C>
struct Vec {
  typedef IO V __attribute__((ext_vector_type(C)));
  typedef V Any __attribute__((aligned(sizeof(IO))));
};
template <typename IO>
struct Vec<IO, 1> {
  typedef IO V;
  typedef IO Any;
};

template <typename IO, int C>
__device__ __forceinline__ typename Vec<IO, C>::V load_any(const IO* p) {
  return *reinterpret_cast<const typename Vec<IO, C>::Any*>(p);
}
template <typename IO, int C>
__device__ __forceinline__ void store_any(IO* p, typename Vec<IO, C>::V v) {
  *reinterpret_cast<typename Vec<IO, C>::Any*>(p) = v;
}

template <int C, typename V>
__device__ __forceinline__ float part(V v, int c) {
  if constexpr (C == 1)
    return float(v);
  else
    return float(v[c]);
}

template <typename IO, int C>
__device__ __forceinline__ typename Vec<IO, C>::V packed(const float (&x)[C]) {
  typename Vec<IO, C>::V v;
  if constexpr (C == 1) {
    v = IO(x[0]);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = IO(x[c]);
  }
  return v;
}

// One token's C channels of an input as they are loaded, or of what was kept of it in 8 bits.
template <typename IO, int C, bool KEPT>
struct In {
  typename Vec<IO, C>::V v;
  __device__ __forceinline__ float get(int c) const { return part<C>(v, c); }
};
template <typename IO, int C>
struct In<IO, C, true> {
  typename Vec<int8_t, C>::V v;
  float scale;
  // a product alone: unsigned bytes and a sum with -128 scales are 2% to 4% faster (gradients of
  // 4 x 4096 x 2048 257 us, so 262; 65536 x 1536 868, so 902), but overflow for a block that
  // holds bfloat16's lowest value
  __device__ __forceinline__ float get(int c) const { return part<C>(v, c) * scale; }
};

// What a tile holds is unpacked again where it is used again: the values of the first use,
// kept as floats, would fill the registers.
template <typename IO, int C, bool KEPT, int T>
__device__ __forceinline__ void as_loaded(In<IO, C, KEPT> (&x)[T]) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    if constexpr (sizeof(x[j].v) >= 4) {
      struct {
        uint32_t w[sizeof(x[j].v) / 4];
      } raw;
      __builtin_memcpy(&raw, &x[j].v, sizeof(raw));
#pragma unroll
      for (uint32_t& w : raw.w) asm("" : "+v"(w));
      __builtin_memcpy(&x[j].v, &raw, sizeof(raw));
    }  // a single narrow value has no copy to save
    if constexpr (KEPT) asm("" : "+v"(x[j].scale));
  }
}

// The tokens of a wave's tile in the order of the scan, and where a row's tokens lie.
struct Span {
  int64_t n, rev, k0;                // tokens of the row, whether it is scanned backwards, the tile's first token
  int live;                          // tokens of the tile that the row has
  __device__ __forceinline__ Span(const RecArgs& a, int64_t b, int64_t first, int tokens) : k0(first) {
    n = a.len;
    if (a.lengths) n = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.len ? a.lengths[b] : a.len;
    rev = a.reverse;
    const int64_t left = n - first;
    live = left <= 0 ? 0 : left < tokens ? int(left) : tokens;
  }
  // where token j of the tile lies; past the row's end, tokens are in their places
  __device__ __forceinline__ int64_t place(int j) const { return rev && k0 + j < n ? n - 1 - (k0 + j) : k0 + j; }
};

// One input's tokens of a tile: a scalar address of the lowest of them, and 32-bit offsets from
// there (the check of the arguments keeps sixteen tokens within 2^32 bytes).  Token j lies
// at(j) tokens above it; where the tile has fewer, its last one stands for those missing.
struct Rows {
  int live, rev;
  __device__ __forceinline__ explicit Rows(const Span& s) : live(s.live), rev(int(s.rev)) {}
  __device__ __forceinline__ unsigned at(int j) const {
    const int k = j < live ? j : live - 1;
    return unsigned(rev ? live - 1 - k : k);
  }
  __device__ __forceinline__ int64_t lowest(const Span& s) const { return s.place(rev ? live - 1 : 0); }
};

template <typename IO, int C, bool KEPT>
struct Loader {
  const char* p;
  unsigned step, lane;
  __device__ __forceinline__ Loader(const RecArgs&, const RecIn& in, const int8_t*, const float*, int64_t b, const Span& s,
                                    int64_t ch)
      : p(static_cast<const char*>(in.p) + (b * in.b + Rows(s).lowest(s) * in.t) * int64_t(sizeof(IO))),
        step(unsigned(in.t) * unsigned(sizeof(IO))), lane(unsigned(ch) * unsigned(sizeof(IO))) {}
  __device__ __forceinline__ In<IO, C, false> row(unsigned k) const {
    return {load_any<IO, C>(reinterpret_cast<const IO*>(p + (k * step + lane)))};
  }
};
template <typename IO, int C>
struct Loader<IO, C, true> {
  const int8_t* p;
  const char* scale;
  unsigned step, lane, scale_step, block;
  __device__ __forceinline__ Loader(const RecArgs& a, const RecIn&, const int8_t* q, const float* s, int64_t b,
                                    const Span& sp, int64_t ch)
      : lane(unsigned(ch)) {
    const int64_t blocks = (a.dim + kPackBlock - 1) / kPackBlock, row = b * a.len + Rows(sp).lowest(sp);
    p = q + row * a.dim;
    scale = reinterpret_cast<const char*>(s + row * blocks);
    step = unsigned(a.dim);
    scale_step = unsigned(blocks * 4);
    block = lane / kPackBlock * 4;
  }
  __device__ __forceinline__ In<IO, C, true> row(unsigned k) const {
    return {load_any<int8_t, C>(p + (k * step + lane)), *reinterpret_cast<const float*>(scale + (k * scale_step + block))};
  }
};

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The segment, row and channels of a block (`number`: shared, for the counter).
struct Tile {
  int seg;
  int64_t b, group;
  static __device__ __forceinline__ Tile of(const TileArgs& p, unsigned* number, bool last_first = false) {
    unsigned unit = blockIdx.x;
    if (p.nseg > 1) {
      if (threadIdx.x == 0) *number = atomicAdd(p.ticket, 1u);
      __syncthreads();
      unit = __builtin_amdgcn_readfirstlane(*number);
    }
    const unsigned rows = unsigned(p.a.batch) * p.groups;  // below 2^24, as all blocks
    const unsigned row = unit % rows;
    const int seg = int(unit / rows);
    return {last_first ? p.nseg - 1 - seg : seg, int64_t(row / p.groups), int64_t(row % p.groups)};
  }
};

// The map of all the block's waves, one after another: their maps lie in LDS (first: the
// lane's first; channel c is 64 floats after the one before), A and H `half` floats apart and
// a wave's `pitch` after the one before.  STEP 1: from the first wave on; -1: from the last.
template <int STEP, int C>
__device__ __forceinline__ void join(const float* first, int half, int pitch, int waves, float (&A)[C], float (&H)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = 1.0f;
    H[c] = 0.0f;
  }
#pragma unroll 1
  for (int v = 0; v < waves; ++v) {
    const float* w = first + (STEP > 0 ? v : waves - 1 - v) * pitch;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float a = w[c * 64];
      H[c] = fmaf(a, H[c], w[c * 64 + half]);
      A[c] *= a;
    }
  }
}

// From the state h that enters the block: puts every wave's entry state in its A's place and
// leaves the exit state in h.
template <int STEP, int C>
__device__ __forceinline__ void hand_on(float* first, int half, int pitch, int waves, float (&h)[C]) {
#pragma unroll 1
  for (int v = 0; v < waves; ++v) {
    float* w = first + (STEP > 0 ? v : waves - 1 - v) * pitch;
    float a[C], b[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      a[c] = w[c * 64];
      b[c] = w[c * 64 + half];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      w[c * 64] = h[c];
      h[c] = fmaf(a[c], h[c], b[c]);
    }
  }
}

template <typename F>
void by_flag(bool v, F f) {
  if (v)
    f(std::true_type());
  else
    f(std::false_type());
}

}  // namespace rec
}  // namespace sscan
