// Dropout, and the root-mean-square norm of a residual stream with its gradients.
//
//   dropout   y = kept ? x * 65536 / (65536 - cut) : 0, kept where the value's 16
//             random bits (psgd_philox.cuh) are not below cut = round(p 65536)
//   norm      r = residual + dropout(x), rounded to the type
//             y = r s w,  s = (mean of r^2 + eps)^-1/2
//   gradient  dr = dr_in + s (dy w - n mean(dy w n)),  n = r s,  dx = dropout(dr)
//             dw = sum over the rows of dy n
//
// All are bound by memory: each value is read once and written once, 16 bytes at
// a time.  Values go in vectors of eight that start at multiples of eight of the
// row-major order, as the random bits do, so a row of odd width is read in
// aligned vectors as well: those at its ends are masked, and what they share with
// the neighbouring rows is written value by value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "psgd_pair.cuh"
#include "psgd_philox.cuh"
#include "psgd_products.h"
#include "psgd_row_vectors.h"

namespace psgd {
namespace {

struct Drop {
  const int64_t* state;  // seed and step; nullptr: no dropout
  uint32_t site, cut;
  float scale;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T of_f(float v);
template <>
__device__ __forceinline__ float of_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 of_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half of_f(float v) { return __float2half_rn(v); }

// Eight values at a 16-byte boundary.
template <typename T>
struct Vec8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* at) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(at) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(T* at) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) __stcs(reinterpret_cast<uint4*>(at) + i, w[i]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const T* t = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f(t[j]);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    T* t = reinterpret_cast<T*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = of_f<T>(v[j]);
  }
};

// ----------------------------------------------------------------- dropout --

template <typename T>
struct DropArgs {
  const T* x;
  T* y;
  int64_t n, cols, ldx, ldy;  // n values; rows of cols where they are not all in a row
  bool flat;                  // in a row, from 16-byte boundaries on
  bool whole;                 // rows of whole vectors, each on such a boundary
  Drop drop;
  int64_t* seen;              // gets the state, or nullptr
};

// Vectors of a thread in flight.  32768 x 8192 bfloat16: 239 us with 1, 190 with 4,
// 166 with 8 (6.5 TB/s, 0.95 of the measured copy), 184 with 16.
constexpr int kDropVecs = 8;

template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs<T> p) {
  grid_wait();
  const Philox bits(p.drop.state, p.drop.site);
  if (p.seen && blockIdx.x == 0 && threadIdx.x < 2) p.seen[threadIdx.x] = p.drop.state[threadIdx.x];
  const int64_t step = (int64_t)gridDim.x * 256, groups = (p.n + 7) / 8, whole = p.flat ? p.n / 8 : 0;
  int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (; g + (kDropVecs - 1) * step < whole; g += kDropVecs * step) {
    Vec8<T> v[kDropVecs];
#pragma unroll
    for (int k = 0; k < kDropVecs; ++k) v[k].load(p.x + (g + k * step) * 8);
#pragma unroll
    for (int k = 0; k < kDropVecs; ++k) {
      float f[8];
      v[k].get(f);
      drop8(f, bits(g + k * step), p.drop.cut, p.drop.scale);
      v[k].set(f);
      v[k].store(p.y + (g + k * step) * 8);
    }
  }
  for (; g < groups; g += step) {
    const int64_t i0 = g * 8;
    float f[8];
    int64_t row = p.flat ? 0 : i0 / p.cols, c = i0 - row * p.cols;
    if (g < whole || p.whole) {
      Vec8<T> v;
      v.load(p.x + row * p.ldx + c);
      v.get(f);
      drop8(f, bits(g), p.drop.cut, p.drop.scale);
      v.set(f);
      v.store(p.y + row * p.ldy + c);
      continue;
    }
    // a last, shorter vector, or rows that start elsewhere: value by value
    const int64_t row0 = row, c0 = c;
    const int count = (int)min((int64_t)8, p.n - i0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = j < count ? to_f(p.x[row * p.ldx + c]) : 0.f;
      if (++c == p.cols) c = 0, ++row;
    }
    drop8(f, bits(g), p.drop.cut, p.drop.scale);
    row = row0, c = c0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < count) p.y[row * p.ldy + c] = of_f<T>(f[j]);
      if (++c == p.cols) c = 0, ++row;
    }
  }
}

// -------------------------------------------------------------------- norm --
//
// A row is held in registers: by four to thirty-two lanes of a warp up to 512
// values, by a CTA up to 8192, by a cluster of CTAs beyond.

constexpr int kMaxWidth = PSGD_MAX_NORM_WIDTH;

template <typename T>
struct NormArgs {
  const T *x, *res;  // forward; gradient: dy and dr_in
  const T* in;       // gradient: r
  T *y, *r;          // gradient: dx and dr
  int64_t ldx, ldres, ldin, ldy, ldr;
  int64_t rows;
  int width;
  int lanes;         // of a warp that share a row
  int ctas;          // of a cluster that share one
  const void* w;     // nullptr: ones
  bool w32;          // float32 weights, whatever T
  float eps;
  Drop drop;
  int64_t* seen;
  float* sums;       // gradient: of each CTA, width values; nullptr: not wanted
};

// A vector of a row that takes lo .. hi - 1 of its eight values.
template <typename T>
__device__ __forceinline__ void load_part(Vec8<T>& v, const T* at, int lo, int hi) {
  if (lo == 0 && hi == 8) {
    v.load(at);
  } else {
    v.zero();
    T* t = reinterpret_cast<T*>(v.w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= lo && j < hi) t[j] = at[j];
  }
}
template <typename T>
__device__ __forceinline__ void store_part(const Vec8<T>& v, T* at, int lo, int hi) {
  if (lo == 0 && hi == 8) {
    v.store(at);
  } else {
    const T* t = reinterpret_cast<const T*>(v.w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= lo && j < hi) at[j] = t[j];
  }
}

// The rows of one thread are a multiple of eight rows apart, so its columns are the same in each of them, wherever rows start
// (ODD: not at vectors): the weight and the sums of its gradient stay in
// registers, kOwnVecs vectors a thread, and the next row's values are asked for
// before the row at hand is reduced.
//
// 2^26 values of bfloat16 with a residual, without dropout, rows of 64 to 8192:
// forward 85-94 us (5.7-6.3 TB/s), gradients 93-116.  Vectors a thread, rows of
// 2048 with dropout: 1 123 and 146 us, 2 93 and 115, 4 114 and 130.  Rows of odd
// width are bound by instructions: 651 130 and 150 us, with dropout 246 and 288;
// rows of clusters by their barrier: 16384 120 and 142 us, 24000 150 and 280.
constexpr int kOwnVecs = 2, kOwnThreads = 512, kOwnCtas = 4;
static_assert((kMaxWidth + 14) / 8 <= kOwnVecs * kOwnThreads * kOwnCtas, "a cluster holds a row");
// Who shares a row.
enum Share { kWarp = 0, kCta = 1, kCluster = 2 };

// Sums of two values over the threads of a row: `lanes` of a warp, the CTA, or
// the cluster, whose CTAs write their warps' sums to each other's shared memory.
// `turn` alternates, so that one barrier a row is enough.
constexpr int kRoom = kOwnThreads / 32 * kOwnCtas;
template <int SHARE>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*room)[kRoom], int turn, int lanes, int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if constexpr (SHARE == kWarp) {
    for (int o = lanes >> 1; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o), b += __shfl_xor_sync(~0u, b, o);
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o), b += __shfl_xor_sync(~0u, b, o);
    if constexpr (SHARE == kCta) {
      if (lane == 0) room[turn][warp] = make_float2(a, b);
      __syncthreads();
      a = b = 0.f;
      for (int w = 0; w < warps; ++w) a += room[turn][w].x, b += room[turn][w].y;
    } else {
      if (lane < ctas) {
        const uint32_t at = map_rank(smem_u32(&room[turn][cluster_rank() * warps + warp]), lane);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
      }
      cluster_sync();
      const int count = ctas * warps;
      const float2 u = lane < count ? room[turn][lane] : make_float2(0.f, 0.f);
      const float2 v = lane + 32 < count ? room[turn][lane + 32] : make_float2(0.f, 0.f);
      a = u.x + v.x, b = u.y + v.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o), b += __shfl_xor_sync(~0u, b, o);
    }
  }
  return make_float2(a, b);
}

// Place of value k of a row's sums: value j of the lanes' vectors in consecutive
// banks, wherever the row starts in its first vector.
__device__ __forceinline__ int place(int k, int pitch) { return (k & 7) * pitch + (k >> 3); }

// A thread's part of the rows: vectors lane, lane + lanes, ... of a row that
// starts at value `off` of its first vector (ODD: not 0 in all of them).  The
// vectors at a row's ends are read whole, and masked; what goes on beside their
// values is kept out of the others' way: with a branch for each of them rows of 651
// bfloat16 values took twice the time.
template <typename T, bool ODD>
struct Span {
  static constexpr int kWords = sizeof(T) == 2 ? 4 : 1;
  int lane, lanes, off, vecs;
  bool in[kOwnVecs], whole[kOwnVecs];  // a vector of the row; with all of its values
  int first[kOwnVecs], end[kOwnVecs];  // the values of it
  bool edge;                           // some vector is not whole
  uint32_t mask[kOwnVecs][kWords];     // 16-bit values: of the row's, in a vector's words
  __device__ __forceinline__ int at(int k) const { return lane + k * lanes; }
  __device__ __forceinline__ void none() {
    edge = false;
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) in[k] = false;
  }
};

template <typename T, bool ODD>
struct RowVecs {
  Vec8<T> v[kOwnVecs];
  // `row`: the row's first vector.  `last`: one of the tensor's last rows, whose last
  // vector ends behind the tensor (first_ragged): only the row's values of it are read.
  __device__ __forceinline__ void load(const T* base, int64_t row, const Span<T, ODD>& s, bool valid, bool last) {
    const T* at = base + row + s.lane * 8;
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) {
      v[k].zero();
      if (s.in[k] && valid && !(ODD && last && s.at(k) == s.vecs - 1)) v[k].load(at + k * s.lanes * 8);
    }
    if (ODD && last && valid) {
#pragma unroll
      for (int k = 0; k < kOwnVecs; ++k)
        if (s.in[k] && s.at(k) == s.vecs - 1) load_part(v[k], at + k * s.lanes * 8, s.first[k], s.end[k]);
    }
  }
  __device__ __forceinline__ void get(int k, float (&f)[8], const Span<T, ODD>& s) const {
    if constexpr (ODD && sizeof(T) == 2) {
      Vec8<T> u;
      u.w[0] = make_uint4(v[k].w[0].x & s.mask[k][0], v[k].w[0].y & s.mask[k][1], v[k].w[0].z & s.mask[k][2],
                          v[k].w[0].w & s.mask[k][3]);
      u.get(f);
    } else {
      v[k].get(f);
      if (ODD && !s.whole[k]) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < s.first[k] || j >= s.end[k]) f[j] = 0.f;
      }
    }
  }
};

// A thread's values of a row.
template <typename T, bool ODD>
__device__ __forceinline__ void store_own(const float (&f)[kOwnVecs][8], T* at, const Span<T, ODD>& s) {
  at += s.lane * 8;
  Vec8<T> v[kOwnVecs];
#pragma unroll
  for (int k = 0; k < kOwnVecs; ++k) {
    v[k].set(f[k]);
    if (s.in[k] && (!ODD || s.whole[k])) v[k].store(at + k * s.lanes * 8);
  }
  if (ODD && s.edge) {
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) {
      if (!s.in[k] || s.whole[k]) continue;
      const T* t = reinterpret_cast<const T*>(v[k].w);
      T* o = at + k * s.lanes * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= s.first[k] && j < s.end[k]) o[j] = t[j];
    }
  }
}

template <typename T, int SHARE, bool ODD>
__device__ __forceinline__ Span<T, ODD> span_of(const NormArgs<T>& p, int64_t row) {
  Span<T, ODD> s;
  s.lanes = SHARE == kWarp ? p.lanes : blockDim.x * (SHARE == kCluster ? p.ctas : 1);
  s.lane = SHARE == kWarp ? threadIdx.x & (p.lanes - 1) : threadIdx.x + (SHARE == kCluster ? cluster_rank() * blockDim.x : 0);
  s.off = ODD ? first_offset(row, p.width) : 0;
  s.vecs = vectors_of(s.off, p.width);
  s.edge = false;
#pragma unroll
  for (int k = 0; k < kOwnVecs; ++k) {
    const int v = s.at(k);
    s.in[k] = v < s.vecs;
    s.first[k] = v ? 0 : s.off, s.end[k] = min(8, s.off + p.width - v * 8);
    s.whole[k] = s.first[k] == 0 && s.end[k] == 8;
    s.edge |= s.in[k] && !s.whole[k];
    if constexpr (ODD && sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < Span<T, ODD>::kWords; ++i)
        s.mask[k][i] = (2 * i >= s.first[k] && 2 * i < s.end[k] ? 0xFFFFu : 0u) |
                       (2 * i + 1 >= s.first[k] && 2 * i + 1 < s.end[k] ? 0xFFFF0000u : 0u);
    }
  }
  return s;
}

template <typename T, bool ODD>
__device__ __forceinline__ void own_weight(const NormArgs<T>& p, float (&w)[kOwnVecs][8], const Span<T, ODD>& s) {
#pragma unroll
  for (int k = 0; k < kOwnVecs; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = s.at(k) * 8 + j - s.off;
      w[k][j] = (unsigned)c >= (unsigned)p.width ? 0.f
                : !p.w                          ? 1.f
                : p.w32                         ? static_cast<const float*>(p.w)[c]
                                                : to_f(static_cast<const T*>(p.w)[c]);
    }
}

template <typename T, int SHARE, bool ODD, bool DROP>
__global__ void __launch_bounds__(SHARE == kWarp ? 256 : kOwnThreads) norm_own_kernel(const NormArgs<T> p) {
  __shared__ float2 room[2][kRoom];
  constexpr bool WARP = SHARE == kWarp;
  const int groups = WARP ? 256 / p.lanes : 1, own = WARP ? threadIdx.x / p.lanes : 0;
  const int block = SHARE == kCluster ? blockIdx.x / p.ctas : blockIdx.x;
  const int64_t step = (int64_t)(SHARE == kCluster ? gridDim.x / p.ctas : gridDim.x) * groups;
  int64_t row = (int64_t)block * groups + own;
  // the warp's rows go together: `ahead` is how far the first of them is in front
  const int ahead = WARP ? (threadIdx.x & 31) / p.lanes : 0;
  if (SHARE == kCluster) cluster_sync();  // the others have started
  grid_wait();
  if (p.seen && blockIdx.x == 0 && threadIdx.x < 2) p.seen[threadIdx.x] = p.drop.state[threadIdx.x];
  Philox bits;
  if (DROP) bits = Philox(p.drop.state, p.drop.site);
  Span<T, ODD> s = span_of<T, SHARE, ODD>(p, row);
  const int64_t ragged = first_ragged(p.rows, p.width);  // ODD: from this row on a last vector ends behind the tensor
  RowVecs<T, ODD> a, b;
  a.load(p.x, row * p.ldx - s.off, s, row < p.rows, row >= ragged);
  if (p.res) b.load(p.res, row * p.ldres - s.off, s, row < p.rows, row >= ragged);
  float w[kOwnVecs][8];
  own_weight(p, w, s);
  const float mean = 1.f / (float)p.width;
  for (int turn = 0; row - ahead < p.rows; row += step, turn ^= 1) {
    if (WARP && row >= p.rows) s.none();
    RowVecs<T, ODD> na, nb;
    const int64_t next = row + step;
    na.load(p.x, next * p.ldx - s.off, s, next < p.rows, next >= ragged);
    if (p.res) nb.load(p.res, next * p.ldres - s.off, s, next < p.rows, next >= ragged);
    float f[kOwnVecs][8], square = 0.f;
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) {
      a.get(k, f[k], s);
      if (DROP) drop8(f[k], bits((uint64_t)(row * p.width - s.off) / 8 + s.at(k)), p.drop.cut, p.drop.scale);
      if (p.res) {
        float g[8];
        b.get(k, g, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] += g[j];
      }
      if (p.r) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] = to_f(of_f<T>(f[k][j]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) square = fmaf(f[k][j], f[k][j], square);
    }
    if (p.r) store_own(f, p.r + (row * p.ldr - s.off), s);
    const float r = rsqrtf(row_sum<SHARE>(square, 0.f, room, turn, s.lanes, p.ctas).x * mean + p.eps);
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[k][j] *= r * w[k][j];
    store_own(f, p.y + (row * p.ldy - s.off), s);
    a = na;
    if (p.res) b = nb;
  }
  if (SHARE == kCluster) cluster_sync();  // no CTA ends while another writes to it
}

template <typename T, int SHARE, bool ODD, bool DROP>
__global__ void __launch_bounds__(SHARE == kWarp ? 256 : kOwnThreads) norm_grad_own_kernel(const NormArgs<T> p) {
  __shared__ float2 room[2][kRoom];
  constexpr bool WARP = SHARE == kWarp;
  constexpr bool kAhead = sizeof(T) == 2;  // float32: no registers for the next row
  const int groups = WARP ? 256 / p.lanes : 1, own = WARP ? threadIdx.x / p.lanes : 0;
  const int block = SHARE == kCluster ? blockIdx.x / p.ctas : blockIdx.x;
  const int64_t step = (int64_t)(SHARE == kCluster ? gridDim.x / p.ctas : gridDim.x) * groups;
  int64_t row = (int64_t)block * groups + own;
  // the warp's rows go together: `ahead` is how far the first of them is in front
  const int ahead = WARP ? (threadIdx.x & 31) / p.lanes : 0;
  if (SHARE == kCluster) cluster_sync();  // the others have started
  grid_wait();
  grid_let_next();
  Philox bits;
  if (DROP) bits = Philox(p.drop.state, p.drop.site);
  Span<T, ODD> s = span_of<T, SHARE, ODD>(p, row);
  const int64_t ragged = first_ragged(p.rows, p.width);  // ODD: from this row on a last vector ends behind the tensor
  RowVecs<T, ODD> a, b, d;
  const auto load = [&](RowVecs<T, ODD>& ra, RowVecs<T, ODD>& rb, RowVecs<T, ODD>& rd, int64_t at) {
    ra.load(p.x, at * p.ldx - s.off, s, at < p.rows, at >= ragged);
    rb.load(p.in, at * p.ldin - s.off, s, at < p.rows, at >= ragged);
    if (p.res) rd.load(p.res, at * p.ldres - s.off, s, at < p.rows, at >= ragged);
  };
  if (kAhead) load(a, b, d, row);
  float w[kOwnVecs][8], sums[kOwnVecs][8];
  own_weight(p, w, s);
#pragma unroll
  for (int k = 0; k < kOwnVecs; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[k][j] = 0.f;
  const float mean = 1.f / (float)p.width;
  for (int turn = 0; row - ahead < p.rows; row += step, turn ^= 1) {
    if (WARP && row >= p.rows) s.none();
    RowVecs<T, ODD> na, nb, nd;
    const int64_t next = row + step;
    if (!kAhead) load(a, b, d, row);
    else load(na, nb, nd, next);
    float square = 0.f, dot = 0.f;
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) {
      float f[8], g[8];
      a.get(k, f, s), b.get(k, g, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) square = fmaf(g[j], g[j], square), dot = fmaf(f[j] * w[k][j], g[j], dot);
    }
    const float2 both = row_sum<SHARE>(square, dot, room, turn, s.lanes, p.ctas);
    // s (dy w - n mean(dy w n)) with n = r s, whose terms stay in range wherever the
    // result does: r s^3 does not, of a row of zeros with a tiny eps or one of 1e15
    const float r = rsqrtf(both.x * mean + p.eps), m = r * (both.y * mean);
    float f[kOwnVecs][8];
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k) {
      float g[8];
      a.get(k, f[k], s), b.get(k, g, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = g[j] * r;
        sums[k][j] = fmaf(f[k][j], n, sums[k][j]);
        f[k][j] = fmaf(-n, m, f[k][j] * w[k][j]) * r;
      }
      if (p.res) {
        d.v[k].get(g);  // beside the row's values anything
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] += g[j];
      }
    }
    if (p.r) store_own(f, p.r + (row * p.ldr - s.off), s);
    if (DROP && p.y) {
#pragma unroll
      for (int k = 0; k < kOwnVecs; ++k)
        drop8(f[k], bits((uint64_t)(row * p.width - s.off) / 8 + s.at(k)), p.drop.cut, p.drop.scale);
      store_own(f, p.y + (row * p.ldy - s.off), s);
    }
    if (kAhead) {
      a = na, b = nb;
      if (p.res) d = nd;
    }
  }
  if (SHARE == kCluster) cluster_sync();
  if (!p.sums) return;
  float* out = p.sums + (int64_t)block * p.width;
  if constexpr (WARP) {  // the sums of the rows' threads, in their order
    const int pitch = p.lanes * kOwnVecs;
    __shared__ float all[256 * kOwnVecs * 8];
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = s.at(k) * 8 + j - s.off;
        if ((unsigned)col < (unsigned)p.width) all[own * pitch * 8 + place(col, pitch)] = sums[k][j];
      }
    __syncthreads();
    for (int col = threadIdx.x; col < p.width; col += 256) {
      float t = 0.f;
      for (int g = 0; g < groups; ++g) t += all[g * pitch * 8 + place(col, pitch)];
      out[col] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kOwnVecs; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = s.at(k) * 8 + j - s.off;
        if ((unsigned)col < (unsigned)p.width) out[col] = sums[k][j];
      }
  }
}

// dw from the CTAs' sums: 32 columns by 32 shares of them a CTA.
template <typename O>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* sums, int count, int width, O* dw, bool add) {
  __shared__ float part[32][32];
  grid_wait();
  const int r = threadIdx.x & 31, g = threadIdx.x >> 5, k = blockIdx.x * 32 + r;
  float t = 0.f;
  if (k < width) {
#pragma unroll 8
    for (int i = g; i < count; i += 32) t += sums[(int64_t)i * width + k];
  }
  part[g][r] = t;
  __syncthreads();
  if (g || k >= width) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) t += part[i][r];
  if (add) t += to_f(dw[k]);
  dw[k] = of_f<O>(t);
}

// ------------------------------------------------------------------- host --

// SMs of the current device, asked once per host thread and device.
int sms_of(int* sms) {
  static thread_local int16_t known[64] = {};
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 64 && known[dev]) {
    *sms = known[dev];
    return PSGD_OK;
  }
  CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  if (dev < 64) known[dev] = (int16_t)*sms;
  return PSGD_OK;
}

// Dropout's arguments; p == 0: none.
int drop_of(double p, const int64_t* state, int site, Drop* d) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(PSGD_ERR_INVALID, "p must be in [0, 1] (got %g)", p);
  if (site < 0 || site > 65535) return fail(PSGD_ERR_INVALID, "site must be in [0, 65535] (got %d)", site);
  *d = Drop{nullptr, (uint32_t)site, (uint32_t)std::lrint(p * 65536.0), 1.f};
  if (!d->cut) return PSGD_OK;
  if (!state || reinterpret_cast<uintptr_t>(state) % 8) return fail(PSGD_ERR_INVALID, "state is NULL or not 8-byte aligned");
  d->state = state;
  d->scale = d->cut == 65536 ? 0.f : (float)(65536.0 / (65536.0 - d->cut));
  return PSGD_OK;
}

int type_size(int dtype) { return dtype == PSGD_F32 ? 4 : 2; }

int check_type(int dtype) {
  return dtype == PSGD_F32 || dtype == PSGD_BF16 || dtype == PSGD_F16 ? PSGD_OK
                                                                     : fail(PSGD_ERR_INVALID, "unknown data type %d", dtype);
}

template <typename T>
int dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, void* y, int64_t ldy, const Drop& d, int64_t* seen,
            cudaStream_t stream) {
  DropArgs<T> a = {};
  a.x = static_cast<const T*>(x), a.y = static_cast<T*>(y), a.n = rows * cols, a.cols = cols, a.ldx = ldx, a.ldy = ldy;
  const bool row = rows == 1 || (ldx == cols && ldy == cols);
  const bool aligned = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % 16 == 0;
  a.flat = row && aligned;
  a.whole = !row && aligned && cols % 8 == 0 && ldx % 8 == 0 && ldy % 8 == 0;
  if (row) a.cols = a.n;
  a.drop = d, a.seen = seen;
  int sms = 0;
  const int rc = sms_of(&sms);
  if (rc) return rc;
  const int64_t ctas = std::min<int64_t>(ceil_div(ceil_div(a.n, 8), 256), sms * 8);
  return launch_behind(dropout_kernel<T>, dim3((unsigned)ctas), 256, 0, stream, a);
}

// Vectors of a row, wherever it starts in its first one.
int most_vecs(int width) { return (width % 8 ? width + 14 : width) / 8; }

constexpr int64_t kMostCtas = 152 * 16;  // of a norm's kernel that stay

// launch_behind for clusters.
template <typename K, typename A>
int launch_cluster(K kernel, dim3 grid, int threads, int ctas, cudaStream_t stream, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.stream = stream;
  cfg.attrs = at, cfg.numAttrs = 2;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args));
  return PSGD_OK;
}

// CTAs of `threads` (whole warps) that an SM holds; asked once per host thread.
template <typename K>
int per_sm(K kernel, int threads, int8_t (&known)[kOwnThreads / 32 + 1], int* per) {
  int8_t& k = known[threads / 32];
  if (!k) {
    CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(per, kernel, threads, 0));
    k = (int8_t)std::max(*per, 1);
  }
  *per = k;
  return PSGD_OK;
}

template <typename T, bool GRAD, int SHARE, bool ODD, bool DROP>
int launch_own(NormArgs<T> a, int sms, int* ctas, cudaStream_t stream) {
  const auto kernel = [] {
    if constexpr (GRAD) return norm_grad_own_kernel<T, SHARE, ODD, DROP>;
    else return norm_own_kernel<T, SHARE, ODD, DROP>;
  }();
  const int vecs = most_vecs(a.width);
  for (a.lanes = 4; SHARE == kWarp && a.lanes * kOwnVecs < vecs;) a.lanes *= 2;
  for (a.ctas = 1; SHARE == kCluster && a.ctas * kOwnVecs * kOwnThreads < vecs;) a.ctas *= 2;  // (3: slower than 4)
  const int threads = SHARE == kWarp ? 256 : (int)(ceil_div(ceil_div(vecs, kOwnVecs * a.ctas), 32) * 32);
  static thread_local int8_t known[kOwnThreads / 32 + 1] = {};
  int per = 0;
  const int rc = per_sm(kernel, threads, known, &per), rows = SHARE == kWarp ? 256 / a.lanes : 1;
  if (rc) return rc;
  // CTAs (or clusters) that stay
  *ctas = (int)std::min<int64_t>({ceil_div(a.rows, rows), (int64_t)(sms / a.ctas) * per, kMostCtas});
  if (ODD && SHARE != kWarp && *ctas < a.rows) *ctas = std::max(8, *ctas / 8 * 8);  // a CTA's rows start alike
  return SHARE == kCluster ? launch_cluster(kernel, dim3((unsigned)(*ctas * a.ctas)), threads, a.ctas, stream, a)
                           : launch_behind(kernel, dim3((unsigned)*ctas), threads, 0, stream, a);
}

template <typename T, bool GRAD, bool ODD, bool DROP>
int launch_rows(const NormArgs<T>& a, int sms, int* ctas, cudaStream_t stream) {
  const int vecs = most_vecs(a.width);
  if (vecs <= 32 * kOwnVecs) return launch_own<T, GRAD, kWarp, ODD, DROP>(a, sms, ctas, stream);
  if (vecs <= kOwnThreads * kOwnVecs) return launch_own<T, GRAD, kCta, ODD, DROP>(a, sms, ctas, stream);
  return launch_own<T, GRAD, kCluster, ODD, DROP>(a, sms, ctas, stream);
}

template <typename T, bool GRAD>
int norm(NormArgs<T> a, int* ctas, cudaStream_t stream) {
  int sms = 0;
  const int rc = sms_of(&sms);
  if (rc) return rc;
  const bool drop = a.drop.cut != 0;
  if (a.width % 8 == 0)
    return drop ? launch_rows<T, GRAD, false, true>(a, sms, ctas, stream) : launch_rows<T, GRAD, false, false>(a, sms, ctas, stream);
  return drop ? launch_rows<T, GRAD, true, true>(a, sms, ctas, stream) : launch_rows<T, GRAD, true, false>(a, sms, ctas, stream);
}

// Rows that the kernels read: 16-byte aligned, and either all in a row or
// whole vectors apart.
int check_rows(const char* name, const void* p, int64_t rows, int64_t ld, int64_t width, int size, bool needed) {
  if (!p && !needed) return PSGD_OK;
  if (!p || reinterpret_cast<uintptr_t>(p) % 16) return fail(PSGD_ERR_INVALID, "%s is NULL or not 16-byte aligned", name);
  if (rows > 1 && (ld < width || ld > ((int64_t)1 << 40) || (ld != width && (ld % 8 || width % 8))))
    return fail(PSGD_ERR_INVALID, "%s: rows of %lld values, %lld apart, are neither in a row nor whole vectors of 8", name,
                (long long)width, (long long)ld);
  return PSGD_OK;
}

int check_norm(int64_t rows, int64_t width, int dtype, const void* w, int w_dtype, float eps) {
  if (rows < 0 || rows > ((int64_t)1 << 40)) return fail(PSGD_ERR_INVALID, "rows must be in [0, 2^40] (got %lld)", (long long)rows);
  if (width < 1 || width > PSGD_MAX_NORM_WIDTH)
    return fail(PSGD_ERR_INVALID, "width must be in [1, %d] (got %lld)", PSGD_MAX_NORM_WIDTH, (long long)width);
  int rc = check_type(dtype);
  if (rc) return rc;
  if (w && w_dtype != PSGD_F32 && w_dtype != dtype)
    return fail(PSGD_ERR_INVALID, "weights are float32 or have the rows' type (got data type %d)", w_dtype);
  if (w && reinterpret_cast<uintptr_t>(w) % type_size(w_dtype)) return fail(PSGD_ERR_INVALID, "the weights are misaligned");
  if (!(eps > 0.f) || std::isinf(eps)) return fail(PSGD_ERR_INVALID, "eps must be positive and finite (got %g)", (double)eps);
  return PSGD_OK;
}

template <typename T>
NormArgs<T> norm_args(int64_t rows, int64_t width, const void* w, int w_dtype, float eps, const Drop& d) {
  NormArgs<T> a = {};
  a.rows = rows, a.width = (int)width, a.w = w, a.w32 = w_dtype == PSGD_F32, a.eps = eps, a.drop = d;
  return a;
}

// Row stride of one row, or of none: any will do.
int64_t stride_of(int64_t rows, int64_t ld, int64_t width) { return rows > 1 ? ld : width; }

template <typename T>
int norm_grad(NormArgs<T> a, void* dw, int dw_dtype, bool add, cudaStream_t stream) {
  int ctas = 0;
  const int rc = norm<T, true>(a, &ctas, stream);
  if (rc || !dw) return rc;
  const dim3 grid((unsigned)ceil_div(a.width, 32));
  const float* sums = a.sums;
  return dw_dtype == PSGD_F32
             ? launch_behind(norm_sums_kernel<float>, grid, 1024, 0, stream, sums, ctas, a.width, static_cast<float*>(dw), add)
             : launch_behind(norm_sums_kernel<T>, grid, 1024, 0, stream, sums, ctas, a.width, static_cast<T*>(dw), add);
}

}  // namespace
}  // namespace psgd

using namespace psgd;

extern "C" int psgd_dropout(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, void* y, int64_t ldy,
                            double p, const int64_t* state, int site, int64_t* seen, void* cuda_stream) {
  int rc = check_type(dtype);
  if (rc) return rc;
  if (rows < 0 || cols < 0 || (cols && rows > ((int64_t)1 << 48) / cols))
    return fail(PSGD_ERR_INVALID, "%lld x %lld is out of range", (long long)rows, (long long)cols);
  Drop d;
  if ((rc = drop_of(p, state, site, &d))) return rc;
  // without dropout the kernel still copies, and needs a state to read
  if (!state || reinterpret_cast<uintptr_t>(state) % 8) return fail(PSGD_ERR_INVALID, "state is NULL or not 8-byte aligned");
  d.state = state;
  if (seen && reinterpret_cast<uintptr_t>(seen) % 8) return fail(PSGD_ERR_INVALID, "seen is not 8-byte aligned");
  if (rows == 0 || cols == 0) return PSGD_OK;
  const int es = type_size(dtype);
  if (!x || !y || (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % es)
    return fail(PSGD_ERR_INVALID, "x or y is NULL or misaligned");
  if (rows > 1 && (ldx < 0 || ldy < cols || ldx > ((int64_t)1 << 40) || ldy > ((int64_t)1 << 40)))
    return fail(PSGD_ERR_INVALID, "row strides %lld and %lld are out of range", (long long)ldx, (long long)ldy);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == PSGD_F32) return dropout<float>(rows, cols, x, ldx, y, ldy, d, seen, s);
  return dtype == PSGD_BF16 ? dropout<__nv_bfloat16>(rows, cols, x, ldx, y, ldy, d, seen, s)
                            : dropout<__half>(rows, cols, x, ldx, y, ldy, d, seen, s);
}

namespace {

template <typename T>
int rms_norm(int64_t rows, int64_t width, const void* x, int64_t ldx, const void* residual, int64_t ldres, const void* w,
             int w_dtype, float eps, const Drop& d, int64_t* seen, void* y, int64_t ldy, void* r, int64_t ldr,
             cudaStream_t s) {
  NormArgs<T> a = norm_args<T>(rows, width, w, w_dtype, eps, d);
  a.x = static_cast<const T*>(x), a.res = static_cast<const T*>(residual), a.y = static_cast<T*>(y), a.r = static_cast<T*>(r);
  a.ldx = stride_of(rows, ldx, width), a.ldres = stride_of(rows, ldres, width);
  a.ldy = stride_of(rows, ldy, width), a.ldr = stride_of(rows, ldr, width);
  a.seen = d.state ? seen : nullptr;
  int ctas;
  return norm<T, false>(a, &ctas, s);
}

template <typename T>
int rms_norm_grad(int64_t rows, int64_t width, const void* dy, int64_t lddy, const void* r, int64_t ldr, const void* dr_in,
                  int64_t lddrin, const void* w, int w_dtype, float eps, const Drop& d, void* dx, int64_t lddx, void* dr,
                  int64_t lddr, void* dw, int dw_dtype, bool add, float* sums, cudaStream_t s) {
  NormArgs<T> a = norm_args<T>(rows, width, w, w_dtype, eps, d);
  a.x = static_cast<const T*>(dy), a.in = static_cast<const T*>(r), a.res = static_cast<const T*>(dr_in);
  a.y = static_cast<T*>(dx), a.r = static_cast<T*>(dr);
  a.ldx = stride_of(rows, lddy, width), a.ldin = stride_of(rows, ldr, width), a.ldres = stride_of(rows, lddrin, width);
  a.ldy = stride_of(rows, lddx, width), a.ldr = stride_of(rows, lddr, width);
  a.sums = dw ? sums : nullptr;
  return norm_grad<T>(a, dw, dw_dtype, add, s);
}

}  // namespace

extern "C" int psgd_rms_norm(int64_t rows, int64_t width, int dtype, const void* x, int64_t ldx, const void* residual,
                             int64_t ldres, const void* w, int w_dtype, float eps, double p, const int64_t* state, int site,
                             int64_t* seen, void* y, int64_t ldy, void* r, int64_t ldr, void* cuda_stream) {
  int rc = check_norm(rows, width, dtype, w, w_dtype, eps);
  Drop d;
  if (rc || (rc = drop_of(p, state, site, &d))) return rc;
  if (seen && reinterpret_cast<uintptr_t>(seen) % 8) return fail(PSGD_ERR_INVALID, "seen is not 8-byte aligned");
  if (rows && !r && (residual || d.cut)) return fail(PSGD_ERR_INVALID, "r must not be NULL with a residual or dropout");
  const int es = type_size(dtype);
  if (rows && ((rc = check_rows("x", x, rows, ldx, width, es, true)) ||
               (rc = check_rows("residual", residual, rows, ldres, width, es, false)) ||
               (rc = check_rows("y", y, rows, ldy, width, es, true)) || (rc = check_rows("r", r, rows, ldr, width, es, false))))
    return rc;
  if (!rows) return PSGD_OK;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const auto f = dtype == PSGD_F32 ? rms_norm<float> : dtype == PSGD_BF16 ? rms_norm<__nv_bfloat16> : rms_norm<__half>;
  return f(rows, width, x, ldx, residual, ldres, w, w_dtype, eps, d, seen, y, ldy, r, ldr, s);
}

extern "C" int psgd_rms_norm_grad(int64_t rows, int64_t width, int dtype, const void* dy, int64_t lddy, const void* r,
                                  int64_t ldr, const void* dr_in, int64_t lddrin, const void* w, int w_dtype, float eps,
                                  double p, const int64_t* state, int site, void* dx, int64_t lddx, void* dr, int64_t lddr,
                                  void* dw, int dw_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                                  void* cuda_stream) {
  int rc = check_norm(rows, width, dtype, w, w_dtype, eps);
  Drop d;
  if (rc || (rc = drop_of(p, state, site, &d))) return rc;
  const int es = type_size(dtype);
  if (dw && ((dw_dtype != PSGD_F32 && dw_dtype != dtype) || reinterpret_cast<uintptr_t>(dw) % type_size(dw_dtype)))
    return fail(PSGD_ERR_INVALID, "dw is float32 or has the rows' type, aligned to it (got data type %d)", dw_dtype);
  if (rows && !dx && !dr && !dw) return fail(PSGD_ERR_INVALID, "the call has no result");
  if (rows && ((rc = check_rows("dy", dy, rows, lddy, width, es, true)) || (rc = check_rows("r", r, rows, ldr, width, es, true)) ||
               (rc = check_rows("dr_in", dr_in, rows, lddrin, width, es, false)) ||
               (rc = check_rows("dx", dx, rows, lddx, width, es, false)) || (rc = check_rows("dr", dr, rows, lddr, width, es, false))))
    return rc;
  const size_t need = dw && rows ? (size_t)std::min<int64_t>(rows, kMostCtas) * width * sizeof(float) : 0;
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < need))
    return fail(PSGD_ERR_INVALID, "the gradient needs a workspace of %zu bytes, 16-byte aligned (got %zu)", need,
                workspace ? workspace_bytes : (size_t)0);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (!rows) {
    if (dw && !accumulate) CUDA_TRY(cudaMemsetAsync(dw, 0, width * type_size(dw_dtype), s));
    return PSGD_OK;
  }
  // without dropout dx is dr
  if (!d.cut && dx) {
    if (dr) return fail(PSGD_ERR_INVALID, "without dropout dx is dr: one of them must be NULL");
    dr = dx, lddr = lddx, dx = nullptr;
  }
  const auto f = dtype == PSGD_F32    ? rms_norm_grad<float>
                 : dtype == PSGD_BF16 ? rms_norm_grad<__nv_bfloat16>
                                      : rms_norm_grad<__half>;
  return f(rows, width, dy, lddy, r, ldr, dr_in, lddrin, w, w_dtype, eps, d, dx, lddx, dr, lddr, dw, dw_dtype, accumulate != 0,
           static_cast<float*>(workspace), s);
}

extern "C" int psgd_rms_norm_workspace(int64_t rows, int64_t width, size_t* bytes) {
  const int rc = check_norm(rows, width, PSGD_F32, nullptr, PSGD_F32, 1.f);
  if (rc) return rc;
  if (!bytes) return fail(PSGD_ERR_INVALID, "bytes must not be NULL");
  *bytes = (size_t)std::min<int64_t>(rows, kMostCtas) * width * sizeof(float);
  return PSGD_OK;
}
