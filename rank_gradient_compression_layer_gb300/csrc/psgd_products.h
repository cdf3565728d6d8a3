// What the operators on the tensor cores share on the host: tensor maps, launches
// that overlap the grid in front, aligned copies of operands that TMA cannot
// read, and the record of products whose kernels gave up a wait.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "psgd_plan.h"

namespace psgd {

// The device's count of abandoned products, made on first use (also while a
// graph is captured).
int abandoned_of(int device, unsigned** count);
// PSGD_ERR_TIMEOUT where products were abandoned that a stream's `waited` call
// (psgd_experts_sync) has not told this thread of, or a product's call nobody.
int report_abandoned(int device, const unsigned* count, cudaStream_t stream, bool waited);
// The limit of a kernel's wait, in units of 1024 ns, and whether this thread's
// products load nothing (psgd_experts_set_wait).
uint32_t wait_limit();
bool wait_stalls();

// A tensor of 16-bit or float32 values (psgd_dtype), innermost dimension first,
// moved in boxes of 128 bytes by `box` (by 1) with the 128-byte swizzle; values
// outside read as 0 and are not written.
int encode(CUtensorMap* map, int dtype, const void* base, int dims, const int64_t* size, const int64_t* stride, int box);

// A single row has no stride of its own: any legal one will do.
inline int64_t tma_stride(int64_t ld, int64_t cols, int64_t rows) { return rows > 1 ? ld : (cols + 7) / 8 * 8; }

// An operand of a product: `count` matrices of rows x cols, ld and stride in values.
struct Operand {
  const void* p;
  int64_t ld, stride;
  int64_t count, rows, cols;
};

// TMA reads rows that start on 16-byte boundaries, a whole number of rows
// from one matrix to the next.
bool tma_reads(const Operand& o);
// Bytes of the copy that it needs otherwise.
size_t copy_bytes(const Operand& o);
// Copies what TMA cannot read into the workspace and points the product at it.
// Of several matrices b, those of experts without rows are left out.  `beside`:
// the copies run beside the grid in front, which must not write the operands,
// from where that one lets them; they end after it.
int make_readable(Operand* a, Operand* b, const int32_t* offsets, unsigned char* ws, cudaStream_t stream,
                  bool beside = false);

// A launch that may overlap the end of the grid in front (grid_wait).
template <typename K, typename... A>
int launch_behind(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
  return PSGD_OK;
}

// Raises a kernel's shared-memory limit, once per host thread and device: the
// call also makes the device's context current on a thread that had none (one
// of torch's backward threads), which the map encoder, a driver call, needs.
template <typename K>
int allow_smem(K kernel, size_t bytes, int dev, uint64_t* done) {
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (*done & bit) return PSGD_OK;
  CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  *done |= bit;
  return PSGD_OK;
}

}  // namespace psgd
