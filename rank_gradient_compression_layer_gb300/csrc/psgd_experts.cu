// Matrix products grouped by expert, with ragged group sizes.
//
// T rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1]-1
// and the matrix W[e] (N x K).
//   forward      y[t]  = W[e(t)] x[t]
//   grad_input   dx[t] = W[e(t)]^T dy[t]
//   grad_weight  dW[e] = sum over e's rows of dy[t] x[t]^T
// Products of bfloat16 or float16 values, float32 sums, one rounding at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/psgd.h"
#include "psgd_pair.cuh"
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
  unsigned char* ws;  // for operands that TMA cannot read
  size_t ws_bytes;
};

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

enum Op { kForward = 0, kGradInput = 1, kGradWeight = 2 };

// ------------------------------------------- pairs of CTAs, tcgen05 + TMA --
//
// The weights' output side is the MMA's M (256 rows a tile), the expert's rows
// (or, for the weight gradient, k) its N, which is chosen per tile: a ragged
// group costs only its own rows, rounded up to 32.
//   forward      D[n, t] = W[n, :] . x[t, :]      A K-major,  B K-major
//   grad_input   D[k, t] = W[:, k] . dy[t, :]     A MN-major, B K-major
//   grad_weight  D[n, k] = dy[:, n] . x[:, k]     A and B MN-major, over e's rows
// Roles of a CTA: warps 0-7 write results (each 32 rows of M by half of the
// columns), warp 8 loads, warp 9 (leader) issues the MMAs, warp 10 (grad_weight)
// clears the rows behind an expert's last one in the last block of its
// contraction.  Two accumulators of 256 columns let the results of a tile go
// out while the next is computed.
//
// The tensor cores truncate each addition: after s instructions a sum is about
// s x 2e-8 of itself too small (4.8e-6 over 4096 rows, where plain float32 has
// 6e-7).  The weight gradient, float32 and as long as an expert has rows,
// therefore takes its sum out of TMEM every kRun blocks (512 rows) and adds
// the pieces in registers, rounded to nearest.  Results of 16 bits do not see it.
constexpr int kStages = 6;
constexpr int kBlock = 64;                     // contraction values of a stage
constexpr int kSideBytes = 128 * kBlock * 2;   // one operand of one CTA and stage
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kChunkBytes = 64 * 128;          // 64 rows of an MN-major operand
constexpr int kBoxRows = 32;                   // rows of one load of the row operand
constexpr int kTileM = 256, kTileN = 256;
constexpr int kPanel = 8;
constexpr int kRun = 8;
constexpr int kWriters = 8;                     // warps that write results
constexpr int kPairThreads = (kWriters + 3) * 32;
constexpr int kPatch = 32 * 32 * 2;             // a warp's staging of 32 x 32 results

__device__ unsigned g_fault;  // a bounded wait ran out (psgd_experts_sync)

struct PairArgs {
  void* out;
  const int32_t* offsets;
  int64_t ldo, o_stride;
  int64_t rows;
  int experts;
  int mdim;   // result values along M
  int ndim;   // grad_weight: along N
  int depth;  // contraction (grad_weight: the expert's rows)
  int tiles;  // grad_weight
  bool aligned;   // 16-byte stores
};

// Shared memory behind the stages.
struct PairShared {
  uint64_t full[kStages], empty[kStages], fix[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int stop;
  int groups;  // experts + 2: rows before the first expert and behind the last
  // then bound[groups + 1] (first row of each group), tile[groups + 1] (its first row tile)
};

size_t pair_smem(int experts) {
  return 1024 + (size_t)kStages * kStageBytes + kWriters * kPatch + sizeof(PairShared) + (size_t)(experts + 3) * 8;
}

__host__ __device__ constexpr int up32(int v) { return (v + 31) & ~31; }

// One tile of the result.
struct Tile2 {
  int expert;     // -1: rows of no expert
  int row0;       // first row (grad_weight: of the expert)
  int m0;         // first value along M
  int n0, count;  // first value along N (rows are counted from row0) and how many
  int width;      // the MMA's N
  int blocks;     // stages of the contraction; 0: the result is zero
  int last;       // contraction values in the last block
};

// The order of mt x nt tiles: panels of kPanel columns, row by row, so that the
// pairs at work share few rows of A and few columns of B.
__device__ __forceinline__ void in_panels(int idx, int mt, int nt, int& m, int& n) {
  const int panel = idx / (kPanel * mt), in = idx - panel * (kPanel * mt);
  const int width = min(kPanel, nt - panel * kPanel);
  m = in / width;
  n = panel * kPanel + (in - m * width);
}

template <int OP>
__device__ __forceinline__ Tile2 tile_at(const PairArgs& p, const PairShared* sh, int idx) {
  const int* bound = reinterpret_cast<const int*>(sh + 1);
  const int mt = (p.mdim + kTileM - 1) / kTileM;
  Tile2 t;
  int depth;
  if (OP == kGradWeight) {
    const int nt = (p.ndim + kTileN - 1) / kTileN;
    const int w = up32((p.ndim + nt - 1) / nt);
    int m, n;
    t.expert = idx / (mt * nt);
    in_panels(idx - t.expert * (mt * nt), mt, nt, m, n);
    t.m0 = m * kTileM;
    t.n0 = n * w;
    t.count = min(w, p.ndim - t.n0);
    t.row0 = bound[t.expert + 1];
    depth = bound[t.expert + 2] - t.row0;
  } else {
    const int* tile = bound + sh->groups + 1;
    int m, tt;
    in_panels(idx, mt, tile[sh->groups], m, tt);
    int lo = 0, hi = sh->groups;  // the last group whose first tile is <= tt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile[mid] <= tt) lo = mid;
      else hi = mid;
    }
    const int c = bound[lo + 1] - bound[lo], nt = (c + kTileN - 1) / kTileN;
    const int w = up32((c + nt - 1) / nt);
    t.expert = lo >= 1 && lo <= p.experts ? lo - 1 : -1;
    t.m0 = m * kTileM;
    t.n0 = (tt - tile[lo]) * w;
    t.count = min(w, c - t.n0);
    t.row0 = bound[lo];
    depth = t.expert < 0 ? 0 : p.depth;
  }
  t.width = up32(t.count);
  t.blocks = (depth + kBlock - 1) / kBlock;
  t.last = depth - (t.blocks - 1) * kBlock;
  return t;
}

// Two float32 results, as bits, in 16 bits each (the first in the low half).
template <typename O>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
  alignas(4) const O v[2] = {from_f<O>(__uint_as_float(a)), from_f<O>(__uint_as_float(b))};
  return *reinterpret_cast<const uint32_t*>(v);
}

// bound[] and tile[] from the offsets: one warp, 32 groups at a time.
__device__ __forceinline__ void scan_groups(const PairArgs& p, PairShared* sh) {
  int* bound = reinterpret_cast<int*>(sh + 1);
  const int E = p.experts, lane = threadIdx.x & 31, rows = (int)p.rows;
  int* tile = bound + E + 3;
  int top = 0, sum = 0;  // of the groups so far: last row's end, row tiles
  int next = lane <= E ? p.offsets[lane] : 0;
  for (int i0 = 0; i0 <= E; i0 += 32) {
    const int i = i0 + lane;
    int end = i <= E ? min(max(next, 0), rows) : 0;
    if (i + 32 <= E) next = p.offsets[i + 32];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(~0u, end, o));  // lanes below o keep their own
    end = max(end, top);
    int begin = __shfl_up_sync(~0u, end, 1);
    if (lane == 0) begin = top;
    const int own = (end - begin + kTileN - 1) / kTileN;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, incl, o);
      incl += lane >= o ? v : 0;
    }
    if (i <= E) bound[1 + i] = end, tile[i] = sum + incl - own;
    top = __shfl_sync(~0u, end, 31);
    sum += __shfl_sync(~0u, incl, 31);
  }
  if (lane == 0) {
    bound[0] = 0, bound[E + 2] = rows;
    tile[E + 1] = sum, tile[E + 2] = sum + (rows - top + kTileN - 1) / kTileN;
    sh->groups = E + 2;
  }
}

template <typename T, typename O, int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const PairArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  PairShared* sh = reinterpret_cast<PairShared*>(smem + kStages * kStageBytes + kWriters * kPatch);
  int* bound = reinterpret_cast<int*>(sh + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kAmn = OP != kForward, kBmn = OP == kGradWeight;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init_count(&sh->full[s], 2), mbar_init_count(&sh->empty[s], 1), mbar_init_count(&sh->fix[s], 1);
    for (int a = 0; a < 2; ++a) mbar_init_count(&sh->acc_full[a], 1), mbar_init_count(&sh->acc_empty[a], 2 * kWriters);
    sh->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWriters + 1) pair_tmem_alloc(&sh->tmem, 512);
  if (warp == kWriters && lane == 0) tma_prefetch_map(&map_a), tma_prefetch_map(&map_b);
  grid_wait();  // from here on the grids in front are done
  if (warp == 0) scan_groups(p, sh);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  const uint32_t tmem = sh->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles =
      OP == kGradWeight ? p.tiles : (bound + sh->groups + 1)[sh->groups] * ((p.mdim + kTileM - 1) / kTileM);
  volatile int* stop = &sh->stop;

  if (warp == kWriters) {
    // ---- loads
    const uint32_t base = smem_u32(smem);
    const uint32_t full0 = map_rank(smem_u32(&sh->full[0]), 0), fix0 = smem_u32(&sh->fix[0]);
    uint32_t s = 0, phase = 1;
    bool ok = true;
    for (int idx = pair; ok && idx < tiles; idx += pairs) {
      const Tile2 t = tile_at<OP>(p, sh, idx);
      const int half = t.width / 2;
      const int boxes = OP == kGradWeight ? (half + 63) / 64 : (half + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = kSideBytes + boxes * (OP == kGradWeight ? kChunkBytes : kBoxRows * 128);
      const int ma = t.m0 + (int)rank * 128, nb = t.n0 + (int)rank * half;
      for (int b = 0; b < t.blocks; ++b) {
        if (!(ok = __all_sync(~0u, pair_wait(&sh->empty[s], phase, stop, &g_fault)))) break;
        const bool ragged = OP == kGradWeight && b == t.blocks - 1 && (t.last & 15);
        const uint32_t bar = (ragged ? fix0 : full0) + s * 8;
        const uint32_t sa = base + s * kStageBytes, sb = sa + kSideBytes;
        const int d = b * kBlock;
        if (elect_one()) {
          if (ragged) {
            mbar_arrive_tx(&sh->fix[s], bytes);
          } else if (rank == 0) {  // both CTAs' bytes; the two arrivals are those of two clearing warps elsewhere
            mbar_arrive_tx(&sh->full[s], 2 * bytes);
            mbar_arrive_local(&sh->full[s]);
          }
          if (OP == kForward) {
            tma_load_3d(sa, &map_a, d, ma, t.expert, bar);
          } else if (OP == kGradInput) {
            tma_load_3d(sa, &map_a, ma, d, t.expert, bar);
            tma_load_3d(sa + kChunkBytes, &map_a, ma + 64, d, t.expert, bar);
          } else {
            tma_load_2d(sa, &map_a, ma, t.row0 + d, bar);
            tma_load_2d(sa + kChunkBytes, &map_a, ma + 64, t.row0 + d, bar);
          }
          if (OP == kGradWeight) {
            tma_load_2d(sb, &map_b, nb, t.row0 + d, bar);
            if (boxes > 1) tma_load_2d(sb + kChunkBytes, &map_b, nb + 64, t.row0 + d, bar);
          } else {
#pragma unroll
            for (int x = 0; x < 128 / kBoxRows; ++x)
              if (x < boxes) tma_load_2d(sb + x * kBoxRows * 128, &map_b, d, t.row0 + nb + x * kBoxRows, bar);
          }
        }
        __syncwarp();
        if (++s == kStages) s = 0, phase ^= 1;
      }
    }
    if (!ok) {  // let the copies in flight land before the CTA's memory goes
      for (const uint64_t t0 = global_ns(); global_ns() - t0 < 20000000ull;) __nanosleep(1000);
    }
  } else if (warp == kWriters + 1) {
    // ---- MMAs
    if (rank == 0) {
      const uint32_t base = smem_u32(smem);
      uint32_t s = 0, phase = 0, n = 0;
      bool ok = true;
      const uint64_t da0 = pair_sdesc(base, kAmn ? kChunkBytes : 16, 1024);
      const uint64_t db0 = pair_sdesc(base + kSideBytes, kBmn ? kChunkBytes : 16, 1024);
      for (int idx = pair; ok && idx < tiles; idx += pairs) {
        const Tile2 t = tile_at<OP>(p, sh, idx);
        const uint32_t idesc = pair_idesc(kBf16, kAmn, kBmn, t.width);
        const int run = OP == kGradWeight ? kRun : t.blocks;
        for (int r0 = 0; ok && r0 < t.blocks; r0 += run, ++n) {
          const uint32_t a = n & 1, d = tmem + a * kTileN;
          if (!(ok = __all_sync(~0u, pair_wait(&sh->acc_empty[a], (n >> 1 & 1) ^ 1, stop, &g_fault)))) break;
          tc_fence_after();
          const int end = min(r0 + run, t.blocks);
          for (int b = r0; b < end; ++b) {
            if (!(ok = __all_sync(~0u, pair_wait(&sh->full[s], phase, stop, &g_fault)))) break;
            if (OP == kGradWeight && b == t.blocks - 1) fence_acquire_cluster();
            tc_fence_after();
            const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
            const int steps = b == t.blocks - 1 ? (t.last + 15) / 16 : kBlock / 16;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBlock / 16; ++k)
                if (k < steps)
                  pair_mma(d, da + k * (kAmn ? 128 : 2), db + k * (kBmn ? 128 : 2), idesc, b > r0 || k > 0);
              pair_commit(&sh->empty[s]);
              if (b == end - 1) pair_commit(&sh->acc_full[a]);
            }
            __syncwarp();
            if (++s == kStages) s = 0, phase ^= 1;
          }
        }
      }
      if (!ok) {
        for (const uint64_t t0 = global_ns(); global_ns() - t0 < 20000000ull;) __nanosleep(1000);
      }
    }
  } else if (warp == kWriters + 2) {
    if (OP == kGradWeight) {  // ---- rows behind the expert's last one
      uint32_t it = 0, phases = 0;
      bool ok = true;
      for (int idx = pair; ok && idx < tiles; idx += pairs) {
        const Tile2 t = tile_at<OP>(p, sh, idx);
        it += t.blocks;
        if (!t.blocks || !(t.last & 15)) continue;
        const int s = (it - 1) % kStages;
        if (!(ok = __all_sync(~0u, pair_wait(&sh->fix[s], phases >> s & 1, stop, &g_fault)))) break;
        phases ^= 1u << s;
        // contraction index i is line i of every chunk, whatever the swizzle
        const int from = t.last * 128, len = ((t.last + 15) / 16 * 16 - t.last) * 128;
        for (int c = 0; c < 2 * kSideBytes / kChunkBytes; ++c)
          for (int i = lane * 16; i < len; i += 512)
            *reinterpret_cast<uint4*>(smem + s * kStageBytes + c * kChunkBytes + from + i) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&sh->full[s]), 0));
      }
    }
  } else {  // ---- results
    uint32_t n = 0;
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .. + 31
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    for (int idx = pair; idx < tiles; idx += pairs) {
      const Tile2 t = tile_at<OP>(p, sh, idx);
      const int m0 = t.m0 + (int)rank * 128 + quarter * 32;
      bool ok = true;
      if (OP == kGradWeight) {
        // columns 128 half .. + 127, in pieces of 16 rows x 32 columns (tmem_ld_16x32)
        float sum[8][16];
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[q][j] = 0.f;
        for (int r0 = 0; r0 < t.blocks; r0 += kRun, ++n) {
          const uint32_t a = n & 1;
          if (!(ok = __all_sync(~0u, pair_wait(&sh->acc_full[a], n >> 1 & 1, stop, &g_fault)))) break;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const int c = half * 128 + (q >> 1) * 32;
            if (c < t.count) {
              uint32_t f[16], g[16];
              tmem_ld_16x32(tmem + a * kTileN + c + lanes, f);
              tmem_ld_16x32(tmem + a * kTileN + c + lanes + (16u << 16), g);
              tmem_wait_ld(f, g);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[q][j] += __uint_as_float(f[j]), sum[q + 1][j] += __uint_as_float(g[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_rank(smem_u32(&sh->acc_empty[a]), 0));
        }
        if (!ok) break;
        O* out = static_cast<O*>(p.out) + t.expert * p.o_stride + t.n0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c0 = half * 128 + (q >> 1) * 32, left = t.count - c0;
          if (left <= 0) continue;
          const int mq = m0 + (q & 1) * 16;
          if (sizeof(O) == 4 && p.aligned && left >= 32) {
            // neighbouring lanes swap halves of two pieces, so that each has 16
            // bytes in a row and four lanes 64 of them
            const bool odd = lane & 1;
            float* o = reinterpret_cast<float*>(out) + c0 + (odd ? 8 : 0) + (lane & 2) * 2;
#pragma unroll
            for (int i = 0; i < 4; i += 2)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float a0 = sum[q][4 * i + 2 * r], a1 = sum[q][4 * i + 2 * r + 1];
                const float b0 = sum[q][4 * i + 4 + 2 * r], b1 = sum[q][4 * i + 4 + 2 * r + 1];
                const float x = __shfl_xor_sync(~0u, odd ? a0 : b0, 1), y = __shfl_xor_sync(~0u, odd ? a1 : b1, 1);
                const int m = mq + lane / 4 + r * 8;
                if (m < p.mdim)
                  *reinterpret_cast<float4*>(o + (int64_t)m * p.ldo + i * 8) =
                      odd ? make_float4(x, y, b0, b1) : make_float4(a0, a1, x, y);
              }
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int m = mq + lane / 4 + r * 8;
              if (m >= p.mdim) continue;
              O* row = out + (int64_t)m * p.ldo + c0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int c = i * 8 + (lane & 3) * 2;
                if (c < left) row[c] = from_f<O>(sum[q][4 * i + 2 * r]);
                if (c + 1 < left) row[c + 1] = from_f<O>(sum[q][4 * i + 2 * r + 1]);
              }
            }
          }
        }
      } else {
        const uint32_t a = n & 1;
        if (t.blocks) {
          if (!__all_sync(~0u, pair_wait(&sh->acc_full[a], n >> 1 & 1, stop, &g_fault))) break;
          tc_fence_after();
        }
        // 32 rows along M by 32 columns at a time, transposed through shared
        // memory: column j is 64 bytes there, its four 16-byte parts in the
        // order part ^ (j / 2 % 4), free of bank conflicts both ways
        const uint32_t patch = smem_u32(smem + kStages * kStageBytes + warp * kPatch);
        const uint32_t put = patch + (lane & 7) * 64 + ((lane >> 3 ^ (lane >> 1 & 3)) * 16);
        const uint4* get = reinterpret_cast<const uint4*>(smem + kStages * kStageBytes + warp * kPatch) + (lane >> 2) * 4 +
                           ((lane & 3) ^ (lane >> 3 & 3));
        O* out = static_cast<O*>(p.out) + (int64_t)(t.row0 + t.n0) * p.ldo + m0;
        const bool whole = p.aligned && m0 + 32 <= p.mdim;
        uint32_t f[16], g[16];
        for (int c = half * 32; c < t.count; c += 64) {
          if (t.blocks) {
            tmem_ld_16x32(tmem + a * kTileN + c + lanes, f);
            tmem_ld_16x32(tmem + a * kTileN + c + lanes + (16u << 16), g);
            tmem_wait_ld(f, g);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = g[j] = 0;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            store_transposed(put + i * 512, pack2<O>(f[4 * i], f[4 * i + 1]), pack2<O>(f[4 * i + 2], f[4 * i + 3]),
                             pack2<O>(g[4 * i], g[4 * i + 1]), pack2<O>(g[4 * i + 2], g[4 * i + 3]));
          __syncwarp();
          if (whole) {
            O* o = out + (int64_t)(c + (lane >> 2)) * p.ldo + (lane & 3) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = get[i * 32];
              if (c + i * 8 + (lane >> 2) < t.count) *reinterpret_cast<uint4*>(o + i * 8 * p.ldo) = v;
            }
          } else if (m0 + lane < p.mdim) {  // a column at a time, a value each lane
            O* o = out + (int64_t)c * p.ldo + lane;
            const O* from = reinterpret_cast<const O*>(smem + kStages * kStageBytes + warp * kPatch) + (lane & 7);
#pragma unroll 8
            for (int j = 0; j < min(32, t.count - c); ++j)
              o[j * p.ldo] = from[j * 32 + ((lane >> 3) ^ (j >> 1 & 3)) * 8];
          }
          __syncwarp();
        }
        if (t.blocks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_rank(smem_u32(&sh->acc_empty[a]), 0));
          ++n;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kWriters + 1) pair_tmem_free(tmem, 512);
}

// ------------------------------------------------------------------- host --

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

// A tensor of 16-bit values, innermost dimension first, loaded in boxes of 64
// values by `box` (by 1) with the 128-byte swizzle; values outside read as 0.
int encode(CUtensorMap* map, int dtype, const void* base, int dims, const int64_t* size, const int64_t* stride, int box) {
  EncodeFn fn;
  const int rc = encoder(&fn);
  if (rc) return rc;
  cuuint64_t gd[3], gs[2];
  const cuuint32_t bd[3] = {64, (cuuint32_t)box, 1}, es[3] = {1, 1, 1};
  for (int i = 0; i < dims; ++i) gd[i] = (cuuint64_t)size[i];
  for (int i = 0; i + 1 < dims; ++i) gs[i] = (cuuint64_t)stride[i] * 2;
  const CUresult r = fn(map, dtype == PSGD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        (cuuint32_t)dims, const_cast<void*>(base), gd, gs, bd, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PSGD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PSGD_OK;
}

// A single row has no stride of its own: any legal one will do.
int64_t tma_stride(int64_t ld, int64_t cols, int64_t rows) { return rows > 1 ? ld : (cols + 7) / 8 * 8; }

template <typename T, typename O, int OP>
int launch_pair(const ProductArgs& p, int dtype, cudaStream_t stream) {
  int dev = 0, sms = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  // before the encoder, a driver call: makes the device's context current on a thread that had none
  auto kernel = pair_kernel<T, O, OP>;
  CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)pair_smem(kMaxExperts)));
  CUtensorMap ma, mb;
  int rc;
  const int64_t lda = tma_stride(p.lda, OP == kForward ? p.k : p.n, p.rows);
  const int64_t acols = OP == kForward ? p.k : p.n;
  if (OP == kGradWeight) {
    const int64_t sa[2] = {p.n, p.rows}, sb[2] = {p.k, p.rows};
    const int64_t ldb = tma_stride(p.ldb, p.k, p.rows);
    if ((rc = encode(&ma, dtype, p.a, 2, sa, &lda, 64)) || (rc = encode(&mb, dtype, p.b, 2, sb, &ldb, 64))) return rc;
  } else {
    const int64_t sw[3] = {p.k, p.n, p.experts}, sr[2] = {acols, p.rows};
    const int64_t ldw = tma_stride(p.ldb, p.k, p.n);
    const int64_t st[2] = {ldw, p.experts > 1 ? p.b_stride : ldw * p.n};
    if ((rc = encode(&ma, dtype, p.b, 3, sw, st, OP == kForward ? 128 : 64)) ||
        (rc = encode(&mb, dtype, p.a, 2, sr, &lda, kBoxRows)))
      return rc;
  }
  PairArgs a;
  a.out = p.c, a.offsets = p.offsets, a.ldo = p.ldc, a.o_stride = p.c_stride, a.rows = p.rows, a.experts = p.experts;
  a.mdim = OP == kGradInput ? p.k : p.n;
  a.ndim = p.k;
  a.depth = OP == kForward ? p.k : p.n;
  const int vec = 16 / sizeof(O);
  a.aligned = reinterpret_cast<uintptr_t>(p.c) % (vec * sizeof(O)) == 0 && p.ldc % vec == 0 && p.c_stride % vec == 0;
  const int64_t mt = ceil_div(a.mdim, kTileM);
  a.tiles = OP == kGradWeight ? (int)(p.experts * mt * ceil_div(p.k, kTileN)) : 0;
  const int64_t most = OP == kGradWeight ? p.experts * mt * ceil_div(p.k, kTileN)
                                         : mt * (p.rows / kTileN + std::min<int64_t>(p.experts + 2, p.rows));
  if (most > INT32_MAX / 2) return fail(PSGD_ERR_INVALID, "the product has too many tiles (%lld)", (long long)most);
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(sms / 2, most));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = pair_smem(p.experts);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, ma, mb, a));
  return PSGD_OK;
}

// ------------------------------------ operands that TMA cannot read as they are --
//
// Rows that do not start on 16-byte boundaries (an odd width, a shifted view,
// a repeated row) are copied into the workspace first, padded to whole 16
// bytes: one pass over the operand, a small part of a product's time.

struct Matrix16 {
  const unsigned char* src;
  uint4* dst;
  const unsigned char *lo, *hi;  // the bytes that belong to the operand
  int64_t ld, stride;            // in bytes: between rows, and between experts' matrices
  int64_t rows;                  // in all
  int per;                       // rows of one matrix
  int cols, vecs;                // values of a row, 16-byte vectors of a copied row
};

// Every thread makes 16-byte vectors of the copy from the two aligned vectors
// around each, joined at the byte where it starts; kCopies of them at a time,
// so that their loads are in flight together.
constexpr int kCopies = 4;
__device__ __forceinline__ void copy_rows(const Matrix16& m) {
  const int64_t n = m.rows * m.vecs, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += step * kCopies) {
    uint4 lo[kCopies], hi[kCopies];
    const unsigned char* at[kCopies];
    int left[kCopies];  // values of the row in the vector; 0 behind the end
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int64_t i = i0 + c * step;
      left[c] = 0;
      lo[c] = hi[c] = make_uint4(0, 0, 0, 0);
      if (i >= n) continue;
      int64_t row, vec;
      if (n < ((int64_t)1 << 32)) {
        row = (uint32_t)i / (uint32_t)m.vecs, vec = (uint32_t)i - (uint32_t)row * (uint32_t)m.vecs;
      } else {
        row = i / m.vecs, vec = i - row * m.vecs;
      }
      const int64_t e = m.per < m.rows ? (uint32_t)row / (uint32_t)m.per : 0;
      at[c] = m.src + e * m.stride + (row - e * m.per) * m.ld + vec * 16;
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
      m.dst[i0 + c * step] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__global__ void __launch_bounds__(256) copy_kernel(const Matrix16 a, const Matrix16 b) {
  grid_let_next();
  if (a.rows) copy_rows(a);
  if (b.rows) copy_rows(b);
}

// An operand of a product: `count` matrices of rows x cols, ld and stride in values.
struct Operand {
  const void* p;
  int64_t ld, stride;
  int64_t count, rows, cols;
};

// TMA reads rows that start on 16-byte boundaries, a whole number of rows
// from one matrix to the next.
bool tma_reads(const Operand& o) {
  if (reinterpret_cast<uintptr_t>(o.p) % 16) return false;
  if (o.rows > 1 && (o.ld % 8 || o.ld < o.cols)) return false;
  const int64_t ld = tma_stride(o.ld, o.cols, o.rows);
  return o.count <= 1 || (o.stride > 0 && o.stride % ld == 0);
}

size_t copy_bytes(const Operand& o) {
  return tma_reads(o) ? 0 : ((size_t)o.count * o.rows * ((o.cols + 7) / 8) * 16 + 255) / 256 * 256;
}

// Copies what TMA cannot read into the workspace and points the product at it.
int make_readable(Operand* a, Operand* b, unsigned char* ws, size_t ws_bytes, cudaStream_t stream) {
  const size_t na = copy_bytes(*a), nb = copy_bytes(*b);
  if (na + nb == 0) return PSGD_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < na + nb)
    return fail(PSGD_ERR_INVALID, "operands whose rows do not start on 16-byte boundaries need a workspace of %zu bytes, "
                "256-byte aligned (got %zu)", na + nb, ws ? ws_bytes : (size_t)0);
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
    m[i].rows = o->count * o->rows, m[i].per = (int)o->rows;
    m[i].cols = (int)o->cols, m[i].vecs = (int)(ld / 8);
    most = std::max(most, m[i].rows * m[i].vecs);
    o->p = to, o->ld = ld, o->stride = ld * o->rows;
  }
  copy_kernel<<<(unsigned)std::min<int64_t>(ceil_div(most, 256 * kCopies), 152 * 8), 256, 0, stream>>>(m[0], m[1]);
  CUDA_TRY(cudaGetLastError());
  return PSGD_OK;
}

template <int OP>
void operands(const ProductArgs& p, Operand* a, Operand* b) {
  *a = Operand{p.a, p.lda, 0, 1, p.rows, OP == kForward ? p.k : p.n};
  *b = OP == kGradWeight ? Operand{p.b, p.ldb, 0, 1, p.rows, p.k}
                         : Operand{p.b, p.ldb, p.b_stride, p.experts, p.n, p.k};
}

// Zeros for the weight gradient of a call without rows.
template <typename O>
__global__ void __launch_bounds__(256) zero_kernel(O* out, int64_t ld, int64_t stride, int n, int k) {
  O* row = out + blockIdx.y * stride + (int64_t)blockIdx.x * ld;
  for (int i = threadIdx.x; i < k; i += 256) row[i] = from_f<O>(0.f);
}

template <typename T, typename O, int OP>
int product(ProductArgs p, int dtype, cudaStream_t s) {
  if (p.rows == 0) {
    if (OP != kGradWeight) return PSGD_OK;
    zero_kernel<O><<<dim3(p.n, p.experts), 256, 0, s>>>(static_cast<O*>(p.c), p.ldc, p.c_stride, p.n, p.k);
    CUDA_TRY(cudaGetLastError());
    return PSGD_OK;
  }
  Operand a, b;
  operands<OP>(p, &a, &b);
  const int rc = make_readable(&a, &b, p.ws, p.ws_bytes, s);
  if (rc) return rc;
  p.a = a.p, p.lda = a.ld, p.b = b.p, p.ldb = b.ld, p.b_stride = b.stride;
  return launch_pair<T, O, OP>(p, dtype, s);
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

int check_stride(int64_t w_stride) {
  if (w_stride < 0 || w_stride > ((int64_t)1 << 40))
    return fail(PSGD_ERR_INVALID, "w: the experts' stride %lld is out of range", (long long)w_stride);
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
                                    void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc || (rc = check_offsets(offsets)) || (rc = check_matrix("x", x, rows, 2, ldx, k, false)) ||
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_stride(w_stride)) || (rc = check_matrix("y", y, rows, 2, ldy, n, true)))
    return rc;
  const ProductArgs p{x, w, y, offsets, ldx, ldw, ldy, w_stride, 0, rows, experts, (int)n, (int)k,
                      static_cast<unsigned char*>(workspace), workspace_bytes};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == PSGD_BF16 ? product<__nv_bfloat16, __nv_bfloat16, kForward>(p, dtype, s)
                            : product<__half, __half, kForward>(p, dtype, s);
}

extern "C" int psgd_experts_grad_input(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* dy,
                                       int64_t lddy, const void* w, int64_t ldw, int64_t w_stride,
                                       const int32_t* offsets, void* dx, int64_t lddx, void* workspace, size_t workspace_bytes,
                                       void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc || (rc = check_offsets(offsets)) || (rc = check_matrix("dy", dy, rows, 2, lddy, n, false)) ||
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_stride(w_stride)) || (rc = check_matrix("dx", dx, rows, 2, lddx, k, true)))
    return rc;
  const ProductArgs p{dy, w, dx, offsets, lddy, ldw, lddx, w_stride, 0, rows, experts, (int)n, (int)k,
                      static_cast<unsigned char*>(workspace), workspace_bytes};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == PSGD_BF16 ? product<__nv_bfloat16, __nv_bfloat16, kGradInput>(p, dtype, s)
                            : product<__half, __half, kGradInput>(p, dtype, s);
}

extern "C" int psgd_experts_grad_weight(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* dy,
                                        int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets,
                                        int out_dtype, void* dw, int64_t lddw, int64_t dw_stride, void* workspace,
                                        size_t workspace_bytes, void* cuda_stream) {
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
  const ProductArgs p{dy, x, dw, offsets, lddy, ldx, lddw, 0, dw_stride, rows, experts, (int)n, (int)k,
                      static_cast<unsigned char*>(workspace), workspace_bytes};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == PSGD_BF16)
    return out_dtype == PSGD_F32 ? product<__nv_bfloat16, float, kGradWeight>(p, dtype, s)
                                 : product<__nv_bfloat16, __nv_bfloat16, kGradWeight>(p, dtype, s);
  return out_dtype == PSGD_F32 ? product<__half, float, kGradWeight>(p, dtype, s) : product<__half, __half, kGradWeight>(p, dtype, s);
}

extern "C" int psgd_experts_workspace(int op, int64_t rows, int experts, int64_t n, int64_t k, const void* a, int64_t lda,
                                      const void* b, int64_t ldb, int64_t b_stride, size_t* bytes) {
  const int rc = check(rows, experts, n, k, PSGD_BF16);
  if (rc) return rc;
  if (op < kForward || op > kGradWeight) return fail(PSGD_ERR_INVALID, "unknown product %d", op);
  if (!bytes) return fail(PSGD_ERR_INVALID, "bytes must not be NULL");
  const ProductArgs p{a, b, nullptr, nullptr, lda, ldb, 0, b_stride, 0, rows, experts, (int)n, (int)k, nullptr, 0};
  Operand oa, ob;
  if (op == kForward) operands<kForward>(p, &oa, &ob);
  else if (op == kGradInput) operands<kGradInput>(p, &oa, &ob);
  else operands<kGradWeight>(p, &oa, &ob);
  *bytes = rows ? copy_bytes(oa) + copy_bytes(ob) : 0;
  return PSGD_OK;
}

extern "C" int psgd_experts_sync(void* cuda_stream) {
  CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)));
  unsigned fault = 0;
  CUDA_TRY(cudaMemcpyFromSymbol(&fault, g_fault, sizeof(fault)));
  if (!fault) return PSGD_OK;
  fault = 0;
  CUDA_TRY(cudaMemcpyToSymbol(g_fault, &fault, sizeof(fault)));
  return fail(PSGD_ERR_TIMEOUT, "an expert product waited past its limit and was abandoned");
}
