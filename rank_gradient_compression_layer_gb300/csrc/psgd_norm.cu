// The global norm of a set of gradients, and clipping by it.
//
//   norm = sqrt(sum over every value g of the set of g^2)
//   c    = min(1, max_norm / (norm + 1e-6)),   out = c g
//
// A set is a table of spans (a contiguous run of values, or rows of equal
// length a stride apart), handed to the kernels as a launch parameter, so no
// table is copied to the device.  The span table describes one set; `groups`
// sets of the same shape (the workers' packed buffers) differ in their base
// addresses and run in the same launch, one norm each.
//
// Sums: a thread squares 64 bytes of a tile in float32 (at most 32 values,
// relative error <= 10 x 2^-24 of a sum of non-negative terms) and adds that to a
// float64 sum of its own; everything after is float64 in a fixed order (lane
// tree, warps, CTAs), so a result does not change from call to call.  A
// float32 sum of squares that leaves [2^-60, 2^126] (values above 1e19, or
// all below 1e-9, whose squares overflow or lose bits) is taken again in
// float64 from the same registers.
//
// Bound by memory: one pass over the set for the norm, a second one for the
// products, since the factor is known only after the last value.  One
// cooperative launch does both: a CTA's last three tiles wait for the factor
// in registers and shared memory (45 MB on the device), the 48 MB before them
// in L2 (evict-last), and the rest is read again.  Three CTAs of 256 threads
// with eight 16-byte loads each keep 98 KB in flight an SM; their held tiles are
// 64 KB each, so no fourth would fit.  Measured, of
// the 6693 GB/s copy rate: norm of four packed LSTM gradients (509 MB) 78 us,
// 0.98; clipping four ResNet-18 gradients (179 MB) 86 us, where a copy of them
// takes 60 and their norm 33; 1.2 billion bfloat16 values 1031 us, where two
// reads and a write at the copy rate take 1083.  A small set takes 5 us (norm)
// or 8 (clipping) on the device.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/psgd.h"
#include "psgd_internal.h"
#include "psgd_plan.h"

namespace psgd {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;          // 16-byte vectors a thread takes of a tile
constexpr int kMaxSpans = 432;    // spans of one launch
constexpr int kFewSpans = 16;     // spans of a launch with a short table
constexpr int kMaxCtas = 1024;    // CTAs (and partial sums) of one group
constexpr int kCtasPerSm = 3;
constexpr int kCounterStep = 32;  // ints between two groups' tile counters
constexpr int kStash = 2;         // tiles of a CTA that the sums leave in shared memory for the products
constexpr int kStashBytes = kStash * kThreads * kVecs * 16;
constexpr int64_t kKeepBytes = 48000000;  // of a set: what the sums leave in L2 for the products

// One run of values: `rows` rows of `cols`, `lds` (`ldd`) values apart in the
// source (destination).  A contiguous run has rows == 1.  Its places are
// numbered with rows `pitch` = cols rounded up to a whole vector apart, so a
// vector of places never spans two rows.
struct Span {
  uint64_t src, dst;   // byte address, or byte offset from the group's base
  int64_t cols;
  int64_t places;      // (rows - 1) * pitch + cols
  int64_t pitch;
  int64_t lds, ldd;
  int32_t step_r, step_c;  // rows and columns that 32 vectors of places make
  int32_t tile0;       // first tile of the span
  int32_t flags;       // kVecSrc, kVecDst, kLinear
};
constexpr int kVecSrc = 1, kVecDst = 2;  // 16-byte loads (stores) are aligned
constexpr int kLinear = 4;               // place p is value p of the source, and readable

template <int S>
struct Table {
  uint64_t src_base[kMaxWorkers], dst_base[kMaxWorkers];
  int32_t spans, tiles;
  int32_t keep;        // tiles in front of the held ones that stay in L2 for the products
  int32_t pad_;
  Span span[S];
};

template <typename T>
struct Type;
template <>
struct Type<float> {
  static constexpr int kVec = 4;
  __device__ static void unpack(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static float get(float v) { return v; }
  __device__ static float put(float v) { return v; }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static void unpack(uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  __device__ static uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Type<__half> {
  static constexpr int kVec = 8;
  __device__ static void unpack(uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
  }
  __device__ static uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ static float get(__half v) { return __half2float(v); }
  __device__ static __half put(float v) { return __float2half_rn(v); }
};

template <typename T>
constexpr int kTile = kThreads * kVecs * Type<T>::kVec;  // values of one tile

// The span of tile t, the last one whose first tile is <= t; `from` is the
// span of an earlier (UP) or later tile, most often still the same.
template <bool UP, int S>
__device__ __forceinline__ int span_of(const Table<S>& tab, int t, int from) {
  int lo = UP ? from : 0, hi = UP ? tab.spans : from + 1;
  if (UP) {
    if (from + 1 == tab.spans || t < tab.span[from + 1].tile0) return from;
  } else {
    if (t >= tab.span[from].tile0) return from;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.span[mid].tile0 <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Row and column of a place.
__device__ __forceinline__ void place_to_rc(const Span& s, int64_t p, int64_t& r, int64_t& c) {
  if (p < ((int64_t)1 << 32) && s.pitch < ((int64_t)1 << 32)) {
    const uint32_t q = (uint32_t)p / (uint32_t)s.pitch;
    r = q, c = (uint32_t)p - q * (uint32_t)s.pitch;
  } else {
    r = p / s.pitch, c = p - r * s.pitch;
  }
}

// Place of this thread's first vector of a tile: a warp takes 4 KB in a row,
// vector v of lane l being number 32 v + l of it.
template <typename T>
__device__ __forceinline__ int64_t first_place(int i) {
  return (int64_t)i * kTile<T> + ((threadIdx.x >> 5) * (32 * kVecs) + (threadIdx.x & 31)) * Type<T>::kVec;
}

// Visits this thread's vectors of tile `i` of a span in order: f(v, inside, r,
// c) for vector v at row r, column c, `inside` the span or behind its end.
template <typename T, typename F>
__device__ __forceinline__ void each_vector(const Span& s, int i, F f) {
  constexpr int V = Type<T>::kVec;
  int64_t p = first_place<T>(i), r = 0, c = p;
  const bool rows = s.places != s.cols;
  if (rows) place_to_rc(s, p, r, c);
#pragma unroll
  for (int v = 0; v < kVecs; ++v, p += 32 * V) {
    f(v, p < s.places, r, c);
    if (rows) {
      r += s.step_r, c += s.step_c;
      if (c >= s.pitch) c -= s.pitch, ++r;
    } else {
      c += 32 * V;
    }
  }
}

// A 16-byte load with an L2 priority: kept longest, or given up first.
__device__ __forceinline__ uint64_t l2_policy(bool last) {
  uint64_t p;
  if (last)
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  else
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load16(const void* at, uint64_t policy) {
  uint4 u;
  asm volatile("ld.global.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(at), "l"(policy)
               : "memory");
  return u;
}

__device__ __forceinline__ uint4 load16_if(bool p, const void* at, uint64_t policy) {
  uint4 u = make_uint4(0, 0, 0, 0);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t@p ld.global.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;\n\t}"
      : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w)
      : "l"(at), "l"(policy), "r"((int)p)
      : "memory");
  return u;
}

// The vector without its values from number `left` on.
template <typename T>
__device__ __forceinline__ uint4 first_values(uint4 u, int left) {
  const int bits = left * (int)(128 / Type<T>::kVec);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = bits - 32 * j;
    w[j] &= b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether tile `i` lies in one run of memory: a contiguous span, or rows whose
// padding belongs to the buffer; and is whole.
template <typename T>
__device__ __forceinline__ bool linear_tile(const Span& s, int i) {
  return (s.flags & kLinear) && (int64_t)(i + 1) * kTile<T> <= s.places;
}

// Column of this thread's first vector of tile `i` of a span of rows.
template <typename T>
__device__ __forceinline__ int first_column(const Span& s, int i) {
  const int64_t p = first_place<T>(i);
  return p < ((int64_t)1 << 32) ? (int)((uint32_t)p % (uint32_t)s.pitch) : (int)(p % s.pitch);
}

// Loads this thread's part of tile `i` of the span; places past a row's end
// or the span's read as 0.
template <typename T>
__device__ __forceinline__ void load_tile(const Span& s, uint64_t base, int i, uint4 (&u)[kVecs], uint64_t policy) {
  constexpr int V = Type<T>::kVec;
  const T* src = reinterpret_cast<const T*>(base + s.src);
  if (linear_tile<T>(s, i) && (s.flags & kVecSrc)) {
    const T* at = src + first_place<T>(i);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) u[v] = load16(at + v * 32 * V, policy);
    if (s.places != s.cols) {
      const int cols = (int)s.cols, pitch = (int)s.pitch;
      int c = first_column<T>(s, i);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (c + V > cols) u[v] = first_values<T>(u[v], cols - c);
        c += s.step_c;
        if (c >= pitch) c -= pitch;
      }
    }
    return;
  }
  // whole vectors first, without a branch between their loads; then the rest value by value
  uint32_t rest = 0;
  each_vector<T>(s, i, [&](int v, bool inside, int64_t r, int64_t c) {
    const bool whole = inside && (s.flags & kVecSrc) && c + V <= s.cols;
    u[v] = load16_if(whole, src + r * s.lds + c, policy);
    rest |= (uint32_t)(inside && !whole) << v;
  });
  if (rest) {
    each_vector<T>(s, i, [&](int v, bool, int64_t r, int64_t c) {
      if (!(rest >> v & 1)) return;
      const T* at = src + r * s.lds + c;
      T part[V];
#pragma unroll
      for (int j = 0; j < V; ++j) part[j] = c + j < s.cols ? at[j] : T(0.f);
      u[v] = *reinterpret_cast<const uint4*>(part);
    });
  }
}

// Stores a warp's 4 KB at an address that is not 16-byte aligned: every lane
// joins the end of its vector to the start of the next one into an aligned 16
// bytes, and the two ends of the 4 KB go out value by value.
template <typename T>
__device__ __forceinline__ void store_shifted(T* at, const uint4 (&u)[kVecs]) {
  constexpr int V = Type<T>::kVec, E = 16 / V;
  const int lane = threadIdx.x & 31;
  unsigned char* base = reinterpret_cast<unsigned char*>(at);  // of the warp's 4 KB
  const int head = 16 - (int)(reinterpret_cast<uintptr_t>(base) & 15);  // bytes before the first aligned place
  const int words = head >> 2, bits = (head & 3) * 8;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    uint32_t w[8] = {u[v].x, u[v].y, u[v].z, u[v].w};
    const uint4 after = v + 1 < kVecs ? u[v + 1 < kVecs ? v + 1 : v] : make_uint4(0, 0, 0, 0);
    const uint32_t n[4] = {after.x, after.y, after.z, after.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // lane 31 goes on with lane 0's next vector
      const uint32_t own = __shfl_down_sync(~0u, w[j], 1), wrap = __shfl_sync(~0u, n[j], 0);
      w[4 + j] = lane == 31 ? wrap : own;
    }
    uint32_t t[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) t[j] = words & 2 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) t[j] = words & 1 ? t[j + 1] : t[j];
    const uint4 o = make_uint4(__funnelshift_r(t[0], t[1], bits), __funnelshift_r(t[1], t[2], bits),
                               __funnelshift_r(t[2], t[3], bits), __funnelshift_r(t[3], t[4], bits));
    if (v + 1 < kVecs || lane < 31) __stcs(reinterpret_cast<uint4*>(base + head + (v * 32 + lane) * 16), o);
  }
  // the first head bytes, and the last 16 - head
  const uint32_t a[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
  const uint32_t b[4] = {u[kVecs - 1].x, u[kVecs - 1].y, u[kVecs - 1].z, u[kVecs - 1].w};
  uint32_t first = 0, last = 0;
  const int byte = lane * E;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = __shfl_sync(~0u, a[j], 0), y = __shfl_sync(~0u, b[j], 31);
    if (byte >> 2 == j) first = x, last = y;
  }
  first >>= (byte & 3) * 8, last >>= (byte & 3) * 8;
  if (byte < 16) {
    unsigned char* end = base + (32 * kVecs - 1) * 16;
    if (E == 4) {
      if (byte < head) *reinterpret_cast<uint32_t*>(base + byte) = first;
      else *reinterpret_cast<uint32_t*>(end + byte) = last;
    } else {
      if (byte < head) *reinterpret_cast<uint16_t*>(base + byte) = (uint16_t)first;
      else *reinterpret_cast<uint16_t*>(end + byte) = (uint16_t)last;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 u, float factor) {
  float f[Type<T>::kVec];
  Type<T>::unpack(u, f);
#pragma unroll
  for (int j = 0; j < Type<T>::kVec; ++j) f[j] *= factor;
  return Type<T>::pack(f);
}

// Stores factor * (this thread's part of tile `i`).
template <typename T>
__device__ __forceinline__ void store_tile(const Span& s, uint64_t base, int i, uint4 (&u)[kVecs], float factor) {
  constexpr int V = Type<T>::kVec;
  T* dst = reinterpret_cast<T*>(base + s.dst);
#pragma unroll
  for (int v = 0; v < kVecs; ++v) u[v] = scaled<T>(u[v], factor);
  if (linear_tile<T>(s, i) && s.places == s.cols) {
    T* at = dst + first_place<T>(i);
    if (s.flags & kVecDst) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) __stcs(reinterpret_cast<uint4*>(at + v * 32 * V), u[v]);
    } else {
      store_shifted(at - (threadIdx.x & 31) * V, u);
    }
    return;
  }
  each_vector<T>(s, i, [&](int v, bool inside, int64_t r, int64_t c) {
    if (!inside) return;
    T* at = dst + r * s.ldd + c;
    if ((s.flags & kVecDst) && c + V <= s.cols) {
      __stcs(reinterpret_cast<uint4*>(at), u[v]);
    } else {
      T part[V];
      *reinterpret_cast<uint4*>(part) = u[v];
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < s.cols) at[j] = part[j];
    }
  });
}

// The float64 sum of squares of one vector, out of line: few calls get here.
template <typename T>
__device__ __noinline__ double wide_squares(uint4 u) {
  float f[Type<T>::kVec];
  Type<T>::unpack(u, f);
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < Type<T>::kVec; ++j) sum += (double)f[j] * (double)f[j];
  return sum;
}

// Sum of squares of a thread's part of a tile (see the note on sums above).
template <typename T>
__device__ __forceinline__ double squares(const uint4 (&u)[kVecs]) {
  constexpr int V = Type<T>::kVec;
  double sum = 0.0;
#pragma unroll
  for (int h = 0; h < kVecs; h += 4) {
    float a[4];
    uint32_t any = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float f[V];
      Type<T>::unpack(u[h + v], f);
      any |= u[h + v].x | u[h + v].y | u[h + v].z | u[h + v].w;
      a[v] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) a[v] = fmaf(f[j], f[j], a[v]);
    }
    const float s = (a[0] + a[1]) + (a[2] + a[3]);
    if (s >= 0x1p-60f && s <= 0x1p126f) {
      sum += (double)s;
    } else if (any) {
#pragma unroll
      for (int v = 0; v < 4; ++v) sum += wide_squares<T>(u[h + v]);
    }
  }
  return sum;
}

// Sum over the CTA, in a fixed order; the result is thread 0's.
__device__ __forceinline__ double block_sum(double d) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) d += part[w];
  }
  return d;
}

// min(1, max_norm / (norm + 1e-6)), NaN where the norm is.
__device__ __forceinline__ float factor_of(double norm, float max_norm) {
  const double c = (double)max_norm / (norm + 1e-6);
  return c > 1.0 ? 1.f : (float)c;
}

// The CTA's tiles are blockIdx.x, + gridDim.x, ...; `n` of them.
template <int S>
__device__ __forceinline__ int tiles_of_cta(const Table<S>& tab) {
  return (tab.tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
}

// Where this thread's vectors of stashed tile `i` are: read by the thread that wrote them.
__device__ __forceinline__ uint4* stash_of(int i) {
  extern __shared__ uint4 stash[];
  return stash + i * kVecs * kThreads + threadIdx.x;
}

// Sum of squares of the CTA's tiles (thread 0's result).  With HOLD, the last
// tile is left in u and the kStash before it in shared memory.
template <typename T, bool HOLD, int S>
__device__ __forceinline__ double sum_tiles(const Table<S>& tab, uint4 (&u)[kVecs]) {
  const uint64_t base = tab.src_base[blockIdx.y];
  const uint64_t first = l2_policy(false), last = l2_policy(true);
  const int n = tiles_of_cta(tab);
  const int held = HOLD ? tab.tiles - (int)gridDim.x * (1 + kStash) : 0;  // first tile that some CTA holds
  double sum = 0.0;
  int at = 0;
  for (int k = 0; k < n; ++k) {
    const int t = blockIdx.x + k * gridDim.x;
    const Span& s = tab.span[at = span_of<true>(tab, t, at)];
    load_tile<T>(s, base, t - s.tile0, u, HOLD && t < held && t >= held - tab.keep ? last : first);
    sum += squares<T>(u);
    if (HOLD && k < n - 1 && k >= n - 1 - kStash) {
      uint4* to = stash_of(n - 2 - k);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) to[v * kThreads] = u[v];
    }
  }
  return block_sum(sum);
}

// The products of the tiles that this CTA's sums held: its last 1 + kStash.
template <typename T, int S>
__device__ __forceinline__ void scale_held(const Table<S>& tab, float factor, uint4 (&u)[kVecs]) {
  const uint64_t dbase = tab.dst_base[blockIdx.y];
  const int n = tiles_of_cta(tab);
  int at = tab.spans - 1;
  for (int k = n - 1; k >= 0 && k >= n - 1 - kStash; --k) {
    const int t = blockIdx.x + k * gridDim.x;
    const Span& s = tab.span[at = span_of<false>(tab, t, at)];
    if (k < n - 1) {
      const uint4* from = stash_of(n - 2 - k);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) u[v] = from[v * kThreads];
    }
    store_tile<T>(s, dbase, t - s.tile0, u, factor);
  }
}

// The products of tiles `count` - 1 .. 0, which the group's CTAs take from a
// common counter, the last ones first: those are still in L2.  (A fixed share
// each left the slowest CTA 14 us behind the fastest at 4 x 45 MB.)
template <typename T, int S>
__device__ __forceinline__ void scale_rest(const Table<S>& tab, int count, float factor, int* taken, uint4 (&u)[kVecs]) {
  __shared__ int next;
  const uint64_t base = tab.src_base[blockIdx.y], dbase = tab.dst_base[blockIdx.y];
  const uint64_t first = l2_policy(false);
  int at = tab.spans - 1;
  if (threadIdx.x == 0) next = atomicAdd(taken, 1);
  __syncthreads();
  for (int i = next; i < count; i = next) {
    const int t = count - 1 - i;
    const Span& s = tab.span[at = span_of<false>(tab, t, at)];
    load_tile<T>(s, base, t - s.tile0, u, first);
    __syncthreads();  // every thread has read `next`
    if (threadIdx.x == 0) next = atomicAdd(taken, 1);
    store_tile<T>(s, dbase, t - s.tile0, u, factor);
    __syncthreads();
  }
}

// The norm of a group from its `n` partial sums (every thread's result).
__device__ __forceinline__ double group_norm(const double* partial, int n) {
  __shared__ double total;
  double d = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) d += __ldcg(partial + i);
  __syncthreads();  // block_sum's memory is free again
  d = block_sum(d);
  if (threadIdx.x == 0) total = sqrt(d);
  __syncthreads();
  return total;
}

// One cooperative launch for a whole set: the sums, a barrier over the grid,
// then the factor and the products.  Groups are blockIdx.y.
template <typename T, int S, bool CLIP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    whole_kernel(const __grid_constant__ Table<S> tab, double* partial, int* counters, float max_norm, float* norm) {
  int* taken = counters + blockIdx.y * kCounterStep;
  if (CLIP && blockIdx.x == 0 && threadIdx.x == 0) *taken = 0;
  uint4 u[kVecs];
  const double sum = sum_tiles<T, CLIP>(tab, u);
  double* mine = partial + (int64_t)blockIdx.y * gridDim.x;
  if (threadIdx.x == 0) mine[blockIdx.x] = sum;
  cooperative_groups::this_grid().sync();
  if (!CLIP && blockIdx.x) return;
  const double total = group_norm(mine, gridDim.x);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[blockIdx.y] = (float)total;
  if (CLIP) {
    const float factor = factor_of(total, max_norm);
    scale_held<T>(tab, factor, u);
    scale_rest<T>(tab, tab.tiles - (int)gridDim.x * (1 + kStash), factor, taken, u);
  }
}

// A set of more spans than one table holds: the sums of one table after
// another, the norm, then the products.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    part_kernel(const __grid_constant__ Table<kMaxSpans> tab, double* partial, int add) {
  uint4 u[kVecs];
  const double sum = sum_tiles<T, false>(tab, u);
  if (threadIdx.x == 0) {
    double* p = partial + (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    *p = add ? *p + sum : sum;
  }
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const double* partial, int ctas, float max_norm, float* norm,
                                                          float* factor) {
  const double total = group_norm(partial + (int64_t)blockIdx.x * ctas, ctas);
  if (threadIdx.x == 0) norm[blockIdx.x] = (float)total, factor[blockIdx.x] = factor_of(total, max_norm);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    scale_kernel(const __grid_constant__ Table<kMaxSpans> tab, const float* factor) {
  const uint64_t base = tab.src_base[blockIdx.y], dbase = tab.dst_base[blockIdx.y];
  const uint64_t first = l2_policy(false);
  const float c = factor[blockIdx.y];
  uint4 u[kVecs];
  int at = 0;
  for (int t = blockIdx.x; t < tab.tiles; t += gridDim.x) {
    const Span& s = tab.span[at = span_of<true>(tab, t, at)];
    load_tile<T>(s, base, t - s.tile0, u, first);
    store_tile<T>(s, dbase, t - s.tile0, u, c);
  }
}

// ------------------------------------------------------------------- host --

int type_size(int dtype) { return dtype == PSGD_F32 ? 4 : 2; }

struct Job {
  int dtype, groups;
  const uint64_t* src_base;  // per group
  const uint64_t* dst_base;  // per group; null: the norm alone
  float max_norm;
  float* norm;
  unsigned char* ws;
  cudaStream_t stream;
  // the workspace: partial sums, factors, tile counters
  double* partial() const { return reinterpret_cast<double*>(ws); }
  float* factor() const { return reinterpret_cast<float*>(partial() + kMaxWorkers * kMaxCtas); }
  int* counters() const { return reinterpret_cast<int*>(factor() + kMaxWorkers); }
};

// The spans of a set come one at a time from `next(i, span)`; false at the end.
struct Source {
  virtual bool next(Span* s) = 0;
  virtual bool done() = 0;  // next() would give nothing
  virtual void restart() = 0;
};

// Fills one launch's table; false when the source had nothing left.
template <int S>
bool fill(Table<S>& tab, const Job& job, Source& src, int64_t tile_values) {
  tab.spans = 0;
  int64_t tiles = 0;
  while (tab.spans < S && tiles < (1 << 30)) {
    Span s;
    if (!src.next(&s)) break;
    s.tile0 = (int32_t)tiles;
    const int64_t step = tile_values / (kVecs * (kThreads / 32));
    s.step_r = (int32_t)(step / s.pitch), s.step_c = (int32_t)(step % s.pitch);
    tiles += (s.places + tile_values - 1) / tile_values;
    tab.span[tab.spans++] = s;
  }
  tab.tiles = (int32_t)tiles;
  tab.keep = (int32_t)(kKeepBytes / (kThreads * kVecs * 16) / job.groups);
  for (int g = 0; g < job.groups; ++g) {
    tab.src_base[g] = job.src_base[g];
    tab.dst_base[g] = job.dst_base ? job.dst_base[g] : 0;
  }
  return tab.spans > 0;
}

template <typename T, int S, bool CLIP>
int launch_whole(const Table<S>& tab, const Job& job, int sms) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeCooperative;
  at.val.cooperative = 1;
  cfg.gridDim = dim3(std::max(1, std::min(std::min(kMaxCtas, tab.tiles), sms * kCtasPerSm / job.groups)), job.groups);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = job.stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  auto kernel = whole_kernel<T, S, CLIP>;
  if (CLIP) {
    cfg.dynamicSmemBytes = kStashBytes;
    CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStashBytes));
  }
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, tab, job.partial(), job.counters(), job.max_norm, job.norm));
  return PSGD_OK;
}

template <typename T>
int run_type(const Job& job, Source& src, int sms) {
  double* partial = job.partial();
  float* factor = job.factor();
  static thread_local Table<kMaxSpans> tab;
  fill(tab, job, src, kTile<T>);
  if (src.done()) {
    if (tab.spans <= kFewSpans) {
      Table<kFewSpans> few;
      std::memcpy(&few, &tab, sizeof(few));
      return job.dst_base ? launch_whole<T, kFewSpans, true>(few, job, sms)
                          : launch_whole<T, kFewSpans, false>(few, job, sms);
    }
    return job.dst_base ? launch_whole<T, kMaxSpans, true>(tab, job, sms)
                        : launch_whole<T, kMaxSpans, false>(tab, job, sms);
  }
  const int ctas = std::max(1, std::min(kMaxCtas, sms * kCtasPerSm / job.groups));
  const dim3 grid(ctas, job.groups);
  int add = 0;
  do {
    part_kernel<T><<<grid, kThreads, 0, job.stream>>>(tab, partial, add++);
  } while (fill(tab, job, src, kTile<T>));
  finish_kernel<<<job.groups, kThreads, 0, job.stream>>>(partial, ctas, job.max_norm, job.norm, factor);
  if (job.dst_base) {
    src.restart();
    while (fill(tab, job, src, kTile<T>)) scale_kernel<T><<<grid, kThreads, 0, job.stream>>>(tab, factor);
  }
  CUDA_TRY(cudaGetLastError());
  return PSGD_OK;
}

int run(const Job& job, Source& src) {
  int dev = 0, sms = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (job.dtype == PSGD_F32) return run_type<float>(job, src, sms);
  if (job.dtype == PSGD_BF16) return run_type<__nv_bfloat16>(job, src, sms);
  return run_type<__half>(job, src, sms);
}

// A list of tensors (absolute addresses, one group).
struct ListSource : Source {
  int count, dtype;
  const void* const* src;
  void* const* dst;
  const int64_t *rows, *cols, *lds, *ldd;
  int at = 0;
  int64_t taken = 0;  // values of tensor `at` that an earlier span has
  bool done() override {
    while (at < count && (cols[at] == 0 || (rows && rows[at] == 0))) ++at;
    return at >= count;
  }
  bool next(Span* s) override {
    if (done()) return false;
    const int es = type_size(dtype), vec = 16 / es;
    const int64_t n = rows ? rows[at] : 1;
    const bool dense = n == 1 || (lds[at] == cols[at] && (!dst || ldd[at] == cols[at]));
    s->src = reinterpret_cast<uint64_t>(src[at]) + taken * es;
    s->dst = dst ? reinterpret_cast<uint64_t>(dst[at]) + taken * es : 0;
    s->cols = (dense ? n * cols[at] : cols[at]) - taken;
    // a run that starts between 16-byte boundaries: the values before the
    // first of them make a span of their own
    const int64_t head = (int64_t)((16 - s->src % 16) % 16) / es;
    const bool cut = dense && head && s->cols > 16 * vec;
    if (cut) s->cols = head;
    s->pitch = (s->cols + vec - 1) / vec * vec;
    s->places = dense ? s->cols : (n - 1) * s->pitch + s->cols;
    s->lds = dense ? 0 : lds[at];
    s->ldd = dense || !dst ? 0 : ldd[at];
    s->flags = (dense ? kLinear : 0) | (s->src % 16 == 0 && s->lds % vec == 0 ? kVecSrc : 0) |
               (s->dst % 16 == 0 && s->ldd % vec == 0 ? kVecDst : 0);
    if (cut) {
      taken = head;
    } else {
      taken = 0;
      ++at;
    }
    return true;
  }
  void restart() override { at = 0, taken = 0; }
};

// The layers of a packed buffer (offsets from the group's base); layers that
// follow each other without padding make one run.
struct PackedSource : Source {
  int layers;
  const int64_t *n, *m;
  int at = 0;
  int64_t off = 0;
  bool done() override { return at >= layers; }
  bool next(Span* s) override {
    if (at >= layers) return false;
    s->flags = kVecSrc | kVecDst | kLinear;
    s->src = s->dst = (uint64_t)off * 4;
    if (m[at] % 4) {  // padded rows
      s->cols = m[at];
      s->pitch = s->lds = s->ldd = (m[at] + 3) / 4 * 4;
      s->places = (n[at] - 1) * s->pitch + s->cols;
      off += n[at] * s->pitch;
      ++at;
      return true;
    }
    int64_t len = 0;
    while (at < layers && m[at] % 4 == 0) {
      const int64_t v = m[at] ? n[at] * m[at] : n[at];
      len += v;
      ++at;
      off += (v + 3) / 4 * 4;
      if (v % 4) break;
    }
    s->cols = s->places = s->pitch = len;
    s->lds = s->ldd = 0;
    return true;
  }
  void restart() override { at = 0, off = 0; }
};

int check_common(const void* norm, const void* workspace, size_t bytes) {
  if (!norm || reinterpret_cast<uintptr_t>(norm) % 4) return fail(PSGD_ERR_INVALID, "norm is NULL or not 4-byte aligned");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16)
    return fail(PSGD_ERR_INVALID, "workspace is NULL or not 16-byte aligned");
  if (bytes < PSGD_GRAD_NORM_WORKSPACE)
    return fail(PSGD_ERR_INVALID, "workspace has %zu bytes, %zu are needed", bytes, (size_t)PSGD_GRAD_NORM_WORKSPACE);
  return PSGD_OK;
}

int check_max_norm(float max_norm) {
  if (!(max_norm >= 0.f)) return fail(PSGD_ERR_INVALID, "max_norm must be >= 0 (got %g)", (double)max_norm);
  return PSGD_OK;
}

int list_job(int count, const void* const* src, void* const* dst, const int64_t* rows, const int64_t* cols,
             const int64_t* lds, const int64_t* ldd, int dtype, float max_norm, float* norm, void* ws, size_t ws_bytes,
             void* stream) {
  if (count < 0) return fail(PSGD_ERR_INVALID, "count must be >= 0 (got %d)", count);
  if (count && (!src || !cols || (rows && (!lds || (dst && !ldd)))))
    return fail(PSGD_ERR_INVALID, "the tensor table must not be NULL");
  if (dtype != PSGD_F32 && dtype != PSGD_BF16 && dtype != PSGD_F16)
    return fail(PSGD_ERR_INVALID, "unknown data type %d", dtype);
  const int es = type_size(dtype);
  for (int i = 0; i < count; ++i) {
    const int64_t n = rows ? rows[i] : 1;
    if (n < 0 || cols[i] < 0 || (cols[i] && n > ((int64_t)1 << 42) / cols[i]))
      return fail(PSGD_ERR_INVALID, "tensor %d: %lld x %lld is out of range", i, (long long)n, (long long)cols[i]);
    if (n == 0 || cols[i] == 0) continue;
    if (!src[i] || reinterpret_cast<uintptr_t>(src[i]) % es)
      return fail(PSGD_ERR_INVALID, "tensor %d is NULL or misaligned", i);
    if (dst && (!dst[i] || reinterpret_cast<uintptr_t>(dst[i]) % es))
      return fail(PSGD_ERR_INVALID, "output %d is NULL or misaligned", i);
    const auto outside = [&](int64_t ld) { return ld < cols[i] || ld > ((int64_t)1 << 31); };
    if (n > 1 && (outside(lds[i]) || (dst && outside(ldd[i]))))
      return fail(PSGD_ERR_INVALID, "tensor %d: row strides must be in [columns, 2^31]", i);
  }
  int rc = check_common(norm, ws, ws_bytes);
  if (rc) return rc;
  ListSource s;
  s.count = count, s.dtype = dtype, s.src = src, s.dst = dst, s.rows = rows, s.cols = cols, s.lds = lds, s.ldd = ldd;
  const uint64_t zero = 0;
  Job job{dtype, 1, &zero, dst ? &zero : nullptr, max_norm, norm, static_cast<unsigned char*>(ws),
          static_cast<cudaStream_t>(stream)};
  return run(job, s);
}

int packed_job(int layers, const int64_t* n, const int64_t* m, int buffers, const float* const* src, float* const* dst,
               float max_norm, float* norms, void* ws, size_t ws_bytes, void* stream) {
  if (layers < 1 || !n || !m) return fail(PSGD_ERR_INVALID, "a set needs at least one layer, and its shapes");
  for (int l = 0; l < layers; ++l)
    if (n[l] < 1 || n[l] > ((int64_t)1 << 30) || m[l] < 0 || m[l] > ((int64_t)1 << 30) ||
        (m[l] && n[l] > ((int64_t)1 << 40) / m[l]))
      return fail(PSGD_ERR_INVALID, "layer %d: %lld x %lld is out of range", l, (long long)n[l], (long long)m[l]);
  if (buffers < 1 || buffers > kMaxWorkers)
    return fail(PSGD_ERR_INVALID, "the number of buffers must be in [1, %d] (got %d)", kMaxWorkers, buffers);
  if (!src) return fail(PSGD_ERR_INVALID, "grad_ptrs must not be NULL");
  uint64_t sb[kMaxWorkers], db[kMaxWorkers];
  for (int g = 0; g < buffers; ++g) {
    sb[g] = reinterpret_cast<uint64_t>(src[g]);
    db[g] = dst ? reinterpret_cast<uint64_t>(dst[g]) : 0;
    if (!sb[g] || sb[g] % 16) return fail(PSGD_ERR_INVALID, "grad_ptrs[%d] is NULL or not 16-byte aligned", g);
    if (dst && (!db[g] || db[g] % 16)) return fail(PSGD_ERR_INVALID, "out_ptrs[%d] is NULL or not 16-byte aligned", g);
  }
  int rc = check_common(norms, ws, ws_bytes);
  if (rc) return rc;
  PackedSource s;
  s.layers = layers, s.n = n, s.m = m;
  Job job{PSGD_F32, buffers, sb, dst ? db : nullptr, max_norm, norms, static_cast<unsigned char*>(ws),
          static_cast<cudaStream_t>(stream)};
  return run(job, s);
}

static_assert(kMaxWorkers * (kMaxCtas * sizeof(double) + sizeof(float) + kCounterStep * sizeof(int)) <=
                  PSGD_GRAD_NORM_WORKSPACE,
              "workspace constant too small");

}  // namespace
}  // namespace psgd

using namespace psgd;

extern "C" int psgd_grad_norm(int count, const void* const* tensors, const int64_t* rows, const int64_t* cols,
                              const int64_t* ld, int dtype, float* norm, void* workspace, size_t workspace_bytes,
                              void* cuda_stream) {
  return list_job(count, tensors, nullptr, rows, cols, ld, nullptr, dtype, 0.f, norm, workspace, workspace_bytes,
                  cuda_stream);
}

extern "C" int psgd_clip_grad_norm(int count, const void* const* tensors, void* const* outputs, const int64_t* rows,
                                   const int64_t* cols, const int64_t* ld, const int64_t* ld_out, int dtype,
                                   float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                                   void* cuda_stream) {
  if (count > 0 && !outputs) return fail(PSGD_ERR_INVALID, "the output table must not be NULL");
  const int rc = check_max_norm(max_norm);
  if (rc) return rc;
  return list_job(count, tensors, outputs, rows, cols, ld, ld_out, dtype, max_norm, norm, workspace, workspace_bytes,
                  cuda_stream);
}

extern "C" int psgd_packed_grad_norm(int num_layers, const int64_t* n, const int64_t* m, int num_buffers,
                                     const float* const* grad_ptrs, float* norms, void* workspace,
                                     size_t workspace_bytes, void* cuda_stream) {
  return packed_job(num_layers, n, m, num_buffers, grad_ptrs, nullptr, 0.f, norms, workspace, workspace_bytes,
                    cuda_stream);
}

extern "C" int psgd_packed_clip_grad_norm(int num_layers, const int64_t* n, const int64_t* m, int num_buffers,
                                          const float* const* grad_ptrs, float* const* out_ptrs, float max_norm,
                                          float* norms, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  if (!out_ptrs) return fail(PSGD_ERR_INVALID, "out_ptrs must not be NULL");
  const int rc = check_max_norm(max_norm);
  if (rc) return rc;
  return packed_job(num_layers, n, m, num_buffers, grad_ptrs, out_ptrs, max_norm, norms, workspace, workspace_bytes,
                    cuda_stream);
}
