// Matrix products grouped by expert, with ragged group sizes.
//
// T rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1]-1
// and the matrix W[e] (N x K).
//   forward      y[t]  = W[e(t)] x[t]
//   grad_input   dx[t] = W[e(t)]^T dy[t]
//   grad_weight  dW[e] = sum over e's rows of dy[t] x[t]^T
// Products of bfloat16 or float16 values, float32 sums, one rounding at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/psgd.h"
#include "psgd_plan.h"

namespace psgd {
namespace {

constexpr int kMaxExperts = PSGD_MAX_EXPERTS;

struct ProductArgs {
  const void* a;  // T rows: x (forward, grad_weight's second side) or dy
  const void* b;  // weights, or grad_weight's x
  void* c;
  const int32_t* offsets;
  int64_t lda, ldb, ldc;     // row strides, in values
  int64_t b_stride, c_stride;  // between experts
  int64_t rows;
  int experts, n, k;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// Offsets as the kernels use them: within [0, rows] and not falling, whatever
// the caller's array holds.
__device__ __forceinline__ int64_t clamp_offset(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

enum Op { kForward = 0, kGradInput = 1, kGradWeight = 2 };
constexpr int kSide = 64, kDepth = 16;

// One CTA per 64 x 64 tile of the result, the two operands' 64 x 16 slices in
// shared memory, 4 x 4 sums a thread.
template <typename T, typename O, int OP>
__global__ void __launch_bounds__(256) simple_kernel(ProductArgs p) {
  __shared__ float sa[kDepth][kSide + 1], sb[kDepth][kSide + 1];
  __shared__ int64_t s_begin, s_end;
  __shared__ int s_expert;
  if (threadIdx.x == 0) {
    // token tiles of the experts in order, then of the rows behind the last
    int64_t tile = OP == kGradWeight ? 0 : blockIdx.x, at = 0;
    int found = -1;
    int64_t b = 0, e = 0;
    for (int i = 0; i <= p.experts + 1; ++i) {
      // i = 0: rows before the first expert; 1..E: experts; E + 1: behind the last
      const int64_t nx = i <= p.experts ? clamp_offset(p.offsets[i], at, p.rows) : p.rows;
      if (OP == kGradWeight) {
        if (i == (int)blockIdx.z + 1) { found = i, b = at, e = nx; break; }
      } else {
        const int64_t tiles = (nx - at + kSide - 1) / kSide;
        if (tile < tiles) { found = i, b = at + tile * kSide, e = b + kSide < nx ? b + kSide : nx; break; }
        tile -= tiles;
      }
      at = nx;
    }
    s_expert = found - 1, s_begin = b, s_end = e;
  }
  __syncthreads();
  const int expert = s_expert;
  if (expert == -2) return;
  const int64_t begin = s_begin, end = s_end;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t j0 = (int64_t)(OP == kGradWeight ? blockIdx.x : blockIdx.y) * kSide;  // column of the result
  const int64_t i0 = OP == kGradWeight ? (int64_t)blockIdx.y * kSide : begin;  // its row
  const bool live = expert >= 0 && expert < p.experts;
  const int64_t depth = !live ? 0 : OP == kForward ? p.k : OP == kGradInput ? p.n : end - begin;
  const int64_t iend = OP == kGradWeight ? p.n : end, jend = OP == kForward ? p.n : p.k;
  const T* A = static_cast<const T*>(p.a);
  const T* B = static_cast<const T*>(p.b) + (OP == kGradWeight || !live ? 0 : expert * p.b_stride);
  float acc[4][4] = {};
  for (int64_t d0 = 0; d0 < depth; d0 += kDepth) {
    for (int q = threadIdx.x; q < kSide * kDepth; q += 256) {
      // the faster index runs along memory
      const int fast = q % (OP == kForward ? kDepth : kSide), slow = q / (OP == kForward ? kDepth : kSide);
      const int da = OP == kGradWeight ? slow : q % kDepth, ia = OP == kGradWeight ? fast : q / kDepth;
      const int db = OP == kForward ? fast : slow, jb = OP == kForward ? slow : fast;
      float va = 0.f, vb = 0.f;
      if (d0 + da < depth && i0 + ia < iend)
        va = to_f(OP == kGradWeight ? A[(begin + d0 + da) * p.lda + i0 + ia] : A[(i0 + ia) * p.lda + d0 + da]);
      if (d0 + db < depth && j0 + jb < jend)
        vb = to_f(OP == kForward      ? B[(j0 + jb) * p.ldb + d0 + db]
                  : OP == kGradInput ? B[(d0 + db) * p.ldb + j0 + jb]
                                     : B[(begin + d0 + db) * p.ldb + j0 + jb]);
      sa[da][ia] = va;
      sb[db][jb] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[d][ty * 4 + i], sb[d][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  O* C = static_cast<O*>(p.c) + (OP == kGradWeight ? expert * p.c_stride : 0);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (i0 + ty * 4 + i < iend && j0 + tx * 4 + j < jend)
        C[(i0 + ty * 4 + i) * p.ldc + j0 + tx * 4 + j] = from_f<O>(acc[i][j]);
}

template <typename T, typename O, int OP>
int launch(const ProductArgs& p, cudaStream_t s) {
  const int64_t cols = OP == kForward ? p.n : p.k;
  const dim3 grid = OP == kGradWeight ? dim3((unsigned)ceil_div(cols, kSide), (unsigned)ceil_div(p.n, kSide), p.experts)
                                      : dim3((unsigned)(ceil_div(p.rows, kSide) + p.experts + 2), (unsigned)ceil_div(cols, kSide));
  simple_kernel<T, O, OP><<<grid, 256, 0, s>>>(p);
  CUDA_TRY(cudaGetLastError());
  return PSGD_OK;
}

int check(int64_t rows, int experts, int64_t n, int64_t k, int dtype) {
  if (rows < 0 || rows > PSGD_MAX_EXPERT_ROWS)
    return fail(PSGD_ERR_INVALID, "rows must be in [0, %lld] (got %lld)", (long long)PSGD_MAX_EXPERT_ROWS, (long long)rows);
  if (experts < 1 || experts > kMaxExperts)
    return fail(PSGD_ERR_INVALID, "experts must be in [1, %d] (got %d)", kMaxExperts, experts);
  if (n < 1 || n > PSGD_MAX_EXPERT_SIDE || k < 1 || k > PSGD_MAX_EXPERT_SIDE)
    return fail(PSGD_ERR_INVALID, "n and k must be in [1, %lld] (got %lld, %lld)", (long long)PSGD_MAX_EXPERT_SIDE,
                (long long)n, (long long)k);
  if (dtype != PSGD_BF16 && dtype != PSGD_F16)
    return fail(PSGD_ERR_INVALID, "the products take bfloat16 or float16 (got data type %d)", dtype);
  return PSGD_OK;
}

// A matrix argument: not NULL where it has values, aligned to its type, and
// rows that do not run into each other (a row stride of 0 repeats one row).
int check_matrix(const char* name, const void* p, int64_t values, int size, int64_t ld, int64_t cols, bool out) {
  if (values && (!p || reinterpret_cast<uintptr_t>(p) % size))
    return fail(PSGD_ERR_INVALID, "%s is NULL or not %d-byte aligned", name, size);
  if (ld < 0 || (out && ld < cols) || ld > ((int64_t)1 << 40))
    return fail(PSGD_ERR_INVALID, "%s: row stride %lld is out of range", name, (long long)ld);
  return PSGD_OK;
}

int check_offsets(const int32_t* offsets) {
  if (!offsets || reinterpret_cast<uintptr_t>(offsets) % 4)
    return fail(PSGD_ERR_INVALID, "offsets is NULL or not 4-byte aligned");
  return PSGD_OK;
}

}  // namespace
}  // namespace psgd

using namespace psgd;

extern "C" int psgd_experts_forward(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* x,
                                    int64_t ldx, const void* w, int64_t ldw, int64_t w_stride, const int32_t* offsets,
                                    void* y, int64_t ldy, void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc || (rc = check_offsets(offsets)) || (rc = check_matrix("x", x, rows, 2, ldx, k, false)) ||
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_matrix("y", y, rows, 2, ldy, n, true)))
    return rc;
  if (rows == 0) return PSGD_OK;
  const ProductArgs p{x, w, y, offsets, ldx, ldw, ldy, w_stride, 0, rows, experts, (int)n, (int)k};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == PSGD_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, kForward>(p, s) : launch<__half, __half, kForward>(p, s);
}

extern "C" int psgd_experts_grad_input(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* dy,
                                       int64_t lddy, const void* w, int64_t ldw, int64_t w_stride,
                                       const int32_t* offsets, void* dx, int64_t lddx, void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc || (rc = check_offsets(offsets)) || (rc = check_matrix("dy", dy, rows, 2, lddy, n, false)) ||
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_matrix("dx", dx, rows, 2, lddx, k, true)))
    return rc;
  if (rows == 0) return PSGD_OK;
  const ProductArgs p{dy, w, dx, offsets, lddy, ldw, lddx, w_stride, 0, rows, experts, (int)n, (int)k};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == PSGD_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, kGradInput>(p, s)
                            : launch<__half, __half, kGradInput>(p, s);
}

extern "C" int psgd_experts_grad_weight(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* dy,
                                        int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets,
                                        int out_dtype, void* dw, int64_t lddw, int64_t dw_stride, void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc) return rc;
  if (out_dtype != PSGD_F32 && out_dtype != dtype)
    return fail(PSGD_ERR_INVALID, "dw is float32 or has the inputs' type (got data type %d)", out_dtype);
  const int os = out_dtype == PSGD_F32 ? 4 : 2;
  if ((rc = check_offsets(offsets)) || (rc = check_matrix("dy", dy, rows, 2, lddy, n, false)) ||
      (rc = check_matrix("x", x, rows, 2, ldx, k, false)) || (rc = check_matrix("dw", dw, 1, os, lddw, k, true)))
    return rc;
  if (experts > 1 && dw_stride < (n - 1) * lddw + k)
    return fail(PSGD_ERR_INVALID, "dw: the experts' matrices overlap (stride %lld)", (long long)dw_stride);
  const ProductArgs p{dy, x, dw, offsets, lddy, ldx, lddw, 0, dw_stride, rows, experts, (int)n, (int)k};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == PSGD_BF16)
    return out_dtype == PSGD_F32 ? launch<__nv_bfloat16, float, kGradWeight>(p, s)
                                 : launch<__nv_bfloat16, __nv_bfloat16, kGradWeight>(p, s);
  return out_dtype == PSGD_F32 ? launch<__half, float, kGradWeight>(p, s) : launch<__half, __half, kGradWeight>(p, s);
}
