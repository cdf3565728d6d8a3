// Host side of the operators on the tensor cores (psgd_products.h), and the
// kernel that copies operands whose rows TMA cannot read.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "psgd_pair.cuh"
#include "psgd_products.h"

namespace psgd {
namespace {

std::atomic<int> g_wait_ms{2000};  // psgd_experts_set_wait
thread_local bool t_stall = false;

// Products that gave up a wait, per device: their kernels count them in mapped
// host memory, where any call can look without waiting.  `told` is the count
// that some call has reported; a thread keeps the count of its own last report
// for each stream that it uses, so that no other caller's report takes its away.
struct Abandoned {
  std::atomic<unsigned*> count{nullptr};
  std::atomic<unsigned> told{0};
};
constexpr int kMaxDevices = 64;
Abandoned g_abandoned[kMaxDevices];
std::mutex g_abandoned_lock;

struct Seen {
  int device;
  cudaStream_t stream;
  unsigned count;
};
constexpr unsigned kSeen = 64;
thread_local Seen t_seen[kSeen];
thread_local unsigned t_seen_used = 0;

// The calling thread's record of a stream; a new one starts at what has been told.
Seen& seen_of(int device, cudaStream_t stream, unsigned told) {
  const unsigned used = std::min(t_seen_used, kSeen);
  for (unsigned i = 0; i < used; ++i)
    if (t_seen[i].device == device && t_seen[i].stream == stream) return t_seen[i];
  Seen& s = t_seen[t_seen_used++ % kSeen];
  s = Seen{device, stream, told};
  return s;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encoder(EncodeFn* fn) {
  static std::atomic<EncodeFn> known{nullptr};
  *fn = known.load(std::memory_order_acquire);
  if (*fn) return PSGD_OK;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q));
  if (q != cudaDriverEntryPointSuccess || !p) return fail(PSGD_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  *fn = reinterpret_cast<EncodeFn>(p);
  known.store(*fn, std::memory_order_release);
  return PSGD_OK;
}

// ------------------------------------ operands that TMA cannot read as they are --
//
// Rows that do not start on 16-byte boundaries (an odd width, a shifted view,
// a repeated row) are copied into the workspace first, padded to whole 16
// bytes: one pass over the operand.  For 5003 rows of 650 and 11 experts of
// 2600 x 650 (50 MB) the copy takes 20 us and the product 25; a product that
// read such rows value by value took 830.

struct Matrix16 {
  const unsigned char* src;
  uint4* dst;
  const unsigned char *lo, *hi;  // the bytes that belong to the operand
  int64_t ld, stride;            // in bytes: between rows, and between experts' matrices
  int64_t rows;                  // of one matrix
  int count;                     // matrices; 0: nothing to copy
  int cols, vecs;                // values of a row, 16-byte vectors of a copied row
};

// Every thread makes 16-byte vectors first, first + step, ... of the copy of
// matrix e from the two aligned vectors around each, joined at the byte where
// it starts; kCopies of them at a time, so that their loads are in flight
// together.
constexpr int kCopies = 4;
__device__ __forceinline__ void copy_rows(const Matrix16& m, int e, int64_t first, int64_t step) {
  const int64_t n = m.rows * m.vecs;
  const unsigned char* src = m.src + e * m.stride;
  uint4* dst = m.dst + e * n;
  for (int64_t i0 = first; i0 < n; i0 += step * kCopies) {
    uint4 lo[kCopies], hi[kCopies];
    const unsigned char* at[kCopies];
    int left[kCopies];  // values of the row in the vector; 0 behind the end
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int64_t i = i0 + c * step;
      left[c] = 0;
      lo[c] = hi[c] = make_uint4(0, 0, 0, 0);
      if (i >= n) continue;
      const int64_t row = n < ((int64_t)1 << 32) ? (uint32_t)i / (uint32_t)m.vecs : i / m.vecs, vec = i - row * m.vecs;
      at[c] = src + row * m.ld + vec * 16;
      left[c] = min(8, m.cols - (int)vec * 8);
      const unsigned char* low = at[c] - (reinterpret_cast<uintptr_t>(at[c]) & 15);
      if (low >= m.lo && low + 32 <= m.hi) {
        lo[c] = *reinterpret_cast<const uint4*>(low);
        hi[c] = *reinterpret_cast<const uint4*>(low + 16);
      } else {  // near an end of the operand: value by value, as if the vector were aligned
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint16_t* v = reinterpret_cast<const uint16_t*>(at[c]) + 2 * j;
          w[j] = (2 * j < left[c] ? (uint32_t)v[0] : 0u) | (2 * j + 1 < left[c] ? (uint32_t)v[1] << 16 : 0u);
        }
        lo[c] = make_uint4(w[0], w[1], w[2], w[3]);
        at[c] = nullptr;
      }
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      if (!left[c]) continue;
      const int shift = (int)(reinterpret_cast<uintptr_t>(at[c]) & 15), bits = (shift & 3) * 8;
      uint32_t w[8] = {lo[c].x, lo[c].y, lo[c].z, lo[c].w, hi[c].x, hi[c].y, hi[c].z, hi[c].w};
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = shift & 8 ? w[j + 2] : w[j];
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = shift & 4 ? w[j + 1] : w[j];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __funnelshift_r(w[j], w[j + 1], bits);
        w[j] = 2 * j + 1 < left[c] ? w[j] : 2 * j < left[c] ? w[j] & 0xFFFFu : 0u;
      }
      dst[i0 + c * step] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// An operand of rows by the whole grid; weights by blockIdx.y = expert, those
// of experts without rows left out.
__global__ void __launch_bounds__(256) copy_kernel(const Matrix16 a, const Matrix16 b, const int32_t* offsets) {
  grid_let_next();
  const int64_t own = (int64_t)blockIdx.x * 256 + threadIdx.x, row = (int64_t)gridDim.x * 256;
  const int64_t all = own + blockIdx.y * row;
  if (a.count) copy_rows(a, 0, all, row * gridDim.y);
  if (b.count == 1) copy_rows(b, 0, all, row * gridDim.y);
  if (b.count > 1 && offsets[blockIdx.y + 1] > offsets[blockIdx.y]) copy_rows(b, blockIdx.y, own, row);
  grid_wait();  // beside another grid: not to end before it
}

}  // namespace

int abandoned_of(int device, unsigned** count) {
  if (device >= kMaxDevices) return fail(PSGD_ERR_INVALID, "more than %d devices", kMaxDevices);
  std::atomic<unsigned*>& known = g_abandoned[device].count;
  if ((*count = known.load(std::memory_order_acquire))) return PSGD_OK;
  const std::lock_guard<std::mutex> lock(g_abandoned_lock);
  if ((*count = known.load(std::memory_order_acquire))) return PSGD_OK;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  CUDA_TRY(cudaThreadExchangeStreamCaptureMode(&mode));
  void* p = nullptr;
  const cudaError_t e = cudaHostAlloc(&p, sizeof(unsigned), cudaHostAllocPortable | cudaHostAllocMapped);
  CUDA_TRY(cudaThreadExchangeStreamCaptureMode(&mode));
  CUDA_TRY(e);
  *count = static_cast<unsigned*>(p);
  **count = 0;
  known.store(*count, std::memory_order_release);
  return PSGD_OK;
}

int report_abandoned(int device, const unsigned* count, cudaStream_t stream, bool waited) {
  std::atomic<unsigned>& told = g_abandoned[device].told;
  const unsigned now = *static_cast<const volatile unsigned*>(count), before = told.load(std::memory_order_relaxed);
  Seen& mine = seen_of(device, stream, before);
  if (now == (waited ? mine.count : before)) return PSGD_OK;
  mine.count = now;
  told.store(now, std::memory_order_relaxed);
  return fail(PSGD_ERR_TIMEOUT, waited ? "a product waited past its limit and was abandoned"
                                       : "an earlier product waited past its limit and was abandoned; nothing was "
                                         "enqueued for this one");
}

uint32_t wait_limit() { return (uint32_t)((uint64_t)g_wait_ms.load(std::memory_order_relaxed) * 1000000u >> 10); }
bool wait_stalls() { return t_stall; }

int encode(CUtensorMap* map, int dtype, const void* base, int dims, const int64_t* size, const int64_t* stride, int box) {
  EncodeFn fn;
  const int rc = encoder(&fn);
  if (rc) return rc;
  cuuint64_t gd[3], gs[2];
  const int size_of = dtype == PSGD_F32 ? 4 : 2;
  const cuuint32_t bd[3] = {(cuuint32_t)(128 / size_of), (cuuint32_t)box, 1}, es[3] = {1, 1, 1};
  for (int i = 0; i < dims; ++i) gd[i] = (cuuint64_t)size[i];
  for (int i = 0; i + 1 < dims; ++i) gs[i] = (cuuint64_t)stride[i] * size_of;
  const CUtensorMapDataType type = dtype == PSGD_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == PSGD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = fn(map, type, (cuuint32_t)dims, const_cast<void*>(base), gd, gs, bd, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PSGD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PSGD_OK;
}

bool tma_reads(const Operand& o) {
  if (reinterpret_cast<uintptr_t>(o.p) % 16) return false;
  if (o.rows > 1 && (o.ld % 8 || o.ld < o.cols)) return false;
  const int64_t ld = tma_stride(o.ld, o.cols, o.rows);
  return o.count <= 1 || (o.stride > 0 && o.stride % ld == 0);
}

size_t copy_bytes(const Operand& o) {
  return tma_reads(o) ? 0 : ((size_t)o.count * o.rows * ((o.cols + 7) / 8) * 16 + 255) / 256 * 256;
}

int make_readable(Operand* a, Operand* b, const int32_t* offsets, unsigned char* ws, cudaStream_t stream, bool beside) {
  const size_t na = copy_bytes(*a), nb = copy_bytes(*b);
  if (na + nb == 0) return PSGD_OK;
  Matrix16 m[2] = {};
  int64_t most = 0;
  for (int i = 0; i < 2; ++i) {
    Operand* o = i ? b : a;
    if (!(i ? nb : na)) continue;
    unsigned char* to = ws + (i ? na : 0);
    const int64_t ld = (o->cols + 7) / 8 * 8;
    m[i].src = static_cast<const unsigned char*>(o->p);
    m[i].dst = reinterpret_cast<uint4*>(to);
    m[i].lo = m[i].src;
    m[i].hi = m[i].src + 2 * ((o->count - 1) * o->stride + (o->rows - 1) * o->ld + o->cols);
    m[i].ld = o->ld * 2, m[i].stride = o->stride * 2;
    m[i].rows = o->rows, m[i].count = (int)o->count;
    m[i].cols = (int)o->cols, m[i].vecs = (int)(ld / 8);
    most = std::max(most, o->rows * m[i].vecs);
    o->p = to, o->ld = ld, o->stride = ld * o->rows;
  }
  const int64_t experts = std::max(1, m[1].count);
  const int64_t most_ctas = experts == 1 ? 152 * 8 : std::max<int64_t>(4, std::min<int64_t>(128, 152 * 32 / experts));
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(most, 256 * kCopies), most_ctas), (unsigned)experts);
  if (beside) return launch_behind(copy_kernel, grid, 256, 0, stream, m[0], m[1], offsets);
  copy_kernel<<<grid, 256, 0, stream>>>(m[0], m[1], offsets);
  CUDA_TRY(cudaGetLastError());
  return PSGD_OK;
}

}  // namespace psgd

using namespace psgd;

extern "C" int psgd_experts_set_wait(int wait_ms, int test_stall) {
  if (wait_ms < 0 || wait_ms > 60000) return fail(PSGD_ERR_INVALID, "wait_ms must be in [0, 60000] (got %d)", wait_ms);
  g_wait_ms.store(wait_ms ? wait_ms : 2000, std::memory_order_relaxed);
  t_stall = test_stall != 0;
  return PSGD_OK;
}

extern "C" int psgd_experts_sync(void* cuda_stream) {
  CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)));
  int dev = 0, rc;
  unsigned* count;
  CUDA_TRY(cudaGetDevice(&dev));
  if ((rc = abandoned_of(dev, &count))) return rc;
  return report_abandoned(dev, count, static_cast<cudaStream_t>(cuda_stream), true);
}
