// Softmax cross entropy of a linear layer over a large vocabulary, without the
// logits in memory, and its gradients, with the exponentials of a chunk of rows there
// in 16 bits.
//
//   l[t, v] = W[v] . x[t] + b[v]        T rows, V words, H values each
//   loss[t] = log sum_v exp(l[t, v]) - l[t, y[t]]
//   d[t, v] = softmax(l[t])[v] - [v = y[t]]
//   dx[t] = g[t] sum_v d[t, v] W[v]     dW[v] = sum_t g[t] d[t, v] x[t]
//   db[v] = sum_t g[t] d[t, v]
// with g[t] the gradient of the reduced loss in loss[t], 0 for ignored rows.
//
// Logits are in units of log 2 from the tensor core's sum on (one FMA with
// log2 e, the bias added in it), so that an exponential is one ex2.
//
// Rows go in chunks.  Of a chunk, one product (stats) reduces every tile of 256
// words to its largest logit and the sum of exponentials beside it, the target
// left out, which makes the loss log1p(sum of the others / target): exact where
// the target takes nearly everything.  A second product (exact) computes the
// logits again and writes d in 16 bits, rounded once from float32, into a buffer
// of the chunk; the other two products read it from there.
//
// In bfloat16, which has float32's range, one product (first) does for both where
// the call is large (kFirstWork): a
// dot product by row gives the target's logit beforehand, and the buffer gets
// e[v] = exp(l[v] - l[y]), whose sum S over v != y gives loss = log1p(S) and the
// target's probability s = 1 / (1 + S).  d[v] = s e[v], and d[y] = -s S; s is left
// to the other operands: dx[t] = g s (sum_v e[v] W[v]), dW[v] = sum_t e[v] (g s x[t]).
// A row of loss above 44 (S >= 2^64) would come near the end of the range, 2^64 of
// which are left to its sums with W and x: its 256 rows go through the two
// products after all.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "psgd_pair.cuh"
#include "psgd_products.h"

namespace psgd {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kIgnored = -1, kOutside = -2;  // column of a row without a target, or with one outside the vocabulary

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

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// d is kept as d * kUp: in float16 a probability below 6e-8 would be lost.
template <typename T>
constexpr float kUp = std::is_same<T, __half>::value ? 16384.f : 1.f;

// ------------------------------------------------------------- the products --
//
// Dense products on pairs of CTAs (psgd_pair.cuh):
//   stats, exact  D[t, v] = x[t, :] . W[v, :]       A and B K-major
//   dx            D[t, h] = d[t, :] . W[:, h]       A K-major, B MN-major
//   dw            D[v, h] = d[:, v] . x[:, h]       A and B MN-major
// M is 256 a tile, N up to 256.  Warps 0-15 write results, four for each quarter of
// the CTA's rows, 64 columns each; warp 16 loads, warp 17 of the leader issues the
// MMAs.  An accumulator is wanted again when one more tile has been computed, which
// of few values (small H) is soon: a warp takes its columns into registers and lets
// it go before it works on them.  2240 rows of 33278 x 650: 57 us without any
// writing; with sums read as they were needed and exponentials through TMA 81; now
// 75, stored from registers (a thread's 32 bytes are a sector), which leaves
// shared memory to six stages.  (Registers that spill: 108, since shared memory
// leaves the first-level cache little room.)
// Gradients leave through 4 KB patches of shared memory (32 rows of 128 bytes,
// swizzled) by TMA, which also cuts them at the matrix's edges.
enum Mode { kStats = 0, kFirst = 1, kExact = 2, kDx = 3, kDw = 4, kDw16 = 5 };  // dw in float32, in 16 bits

constexpr int kBlock = 64;                     // contraction values of a stage
constexpr int kSideBytes = 128 * kBlock * 2;   // one operand of one CTA and stage
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kChunkBytes = 64 * 128;          // 64 rows of an MN-major operand
constexpr int kTile = 256;
constexpr int kPanel = 8;
constexpr int kWriters = 16, kShares = kWriters / 4;
constexpr int kThreads = (kWriters + 2) * 32;
constexpr int kPatchBytes = 4096;
// Blocks that a sum of dw stays in the tensor core for, at most.  An instruction cuts
// each of the 17 terms that it adds: of operands of one sign that is up to 2.1e-7 of the
// sum, 1.3e-3 over 200000 rows.  The products over the rows, whose results may be
// float32, therefore leave it after 1024 rows (float16) or 2048 (bfloat16, whose
// products of 16 bits are cut later), and are added in registers, rounded to nearest:
// off by 6.2e-6 and 1.8e-7 of a sum of one sign, however many rows.  2240 rows of 33278 x
// 650 bfloat16 take 271 us so, 270 without.
template <typename T>
constexpr int kRun = std::is_same<T, __half>::value ? 16 : 32;
template <int MODE>
constexpr int kStages = MODE <= kExact ? 6 : 5;
template <int MODE>
constexpr int kPatchesOf = MODE <= kExact ? 0 : 1;  // of a warp
template <int MODE>
constexpr int kBiasBytes = MODE <= kExact ? 64 * 4 : 0;  // of a warp's columns

struct DenseArgs {
  int mdim, ndim, depth;  // D is mdim x ndim, a contraction of depth values
  int mt, nt, width;      // tiles, and columns of one
  int parts;              // dx, dw: cuts of the contraction, each with sums of its own
  int64_t part_rows;      // rows of out between them
  int out_cols;           // dx, dw: columns of out that TMA writes
  // stats and exact
  const int32_t* cols;    // target of each row, kIgnored or kOutside
  const float* bias;      // bias in units of log 2, -inf behind the vocabulary; nullptr: none
  float *top, *sum;       // [kShares tile + share][ld]: largest logit (stats) and sum of the exponentials
  const float* losses;    // exact
  int ld;
  const float* lse;       // exact: log2 of the sum of exponentials; first: the target's logit
  const int* flags;       // rows of tiles that are taken; nullptr: all
  // dw
  const float* scale;     // of the sums
  void* out;              // first, exact: the exponentials' buffer, rows of whole 128 bytes.  dw: its columns
                          // out_cols .. out_end - 1 are written by threads: TMA writes whole
  int64_t ldo;            // 16 bytes, into what lies behind a row, and only rows on such boundaries
  int out_end;
  bool even;              // 16 bits: two values at a time
  float* db;              // sums of column ndim - 1, one part after the other (part_rows apart); nullptr: none
  void* db_out;           // the same in its own type, where nothing is added; db32: float32
  bool db32;
  bool add, db_add;       // to what out and db hold
  bool beside;            // dx: runs beside the grid in front, and ends after it
  bool stall;
  uint32_t wait;
  unsigned* abandoned;
  int* lost;              // set where a wait ran out
};

struct DenseShared {
  uint64_t full[6], empty[6], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int stop;
};

template <int MODE>
constexpr size_t dense_smem() {
  return 1024 + (size_t)kStages<MODE> * kStageBytes + kWriters * (kPatchesOf<MODE> * kPatchBytes + kBiasBytes<MODE>) + sizeof(DenseShared);
}
static_assert(dense_smem<kExact>() <= 232448 && dense_smem<kStats>() <= 232448, "too large");

struct Unit {
  int m0, n0, part, d0, blocks;
  int run;  // blocks that are summed in one go
  int tile_n;
};

template <typename T, int MODE>
__device__ __forceinline__ Unit unit_at(const DenseArgs& p, int idx) {
  Unit u;
  const int q = idx / p.parts;
  u.part = idx - q * p.parts;
  const int panel = q / (kPanel * p.mt), in = q - panel * (kPanel * p.mt);
  const int wide = min(kPanel, p.nt - panel * kPanel);
  const int m = in / wide;
  u.tile_n = panel * kPanel + (in - m * wide);
  u.m0 = m * kTile;
  u.n0 = u.tile_n * p.width;
  const int blocks = (p.depth + kBlock - 1) / kBlock;
  const int b0 = (int)((int64_t)blocks * u.part / p.parts), b1 = (int)((int64_t)blocks * (u.part + 1) / p.parts);
  u.d0 = b0 * kBlock;
  u.blocks = b1 - b0;
  const int runs = (u.blocks + kRun<T> - 1) / kRun<T>;
  u.run = MODE < kDw ? u.blocks : (u.blocks + runs - 1) / runs;  // of equal length
  return u;
}

// A patch of shared memory to a tensor, or added to it (float32).
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
               "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_add_2d(const void* map, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's stores still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void put16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float4 get16(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// 32 sums of a row, there after take_sums.
__device__ __forceinline__ void ask_sums(uint32_t from, float (&f)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]),
        "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15]), "=f"(f[16]),
        "=f"(f[17]), "=f"(f[18]), "=f"(f[19]), "=f"(f[20]), "=f"(f[21]), "=f"(f[22]), "=f"(f[23]), "=f"(f[24]),
        "=f"(f[25]), "=f"(f[26]), "=f"(f[27]), "=f"(f[28]), "=f"(f[29]), "=f"(f[30]), "=f"(f[31])
      : "r"(from)
      : "memory");
}
__device__ __forceinline__ void hold32(float (&f)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 16)
    asm volatile(""
                 : "+f"(f[i]), "+f"(f[i + 1]), "+f"(f[i + 2]), "+f"(f[i + 3]), "+f"(f[i + 4]), "+f"(f[i + 5]), "+f"(f[i + 6]),
                   "+f"(f[i + 7]), "+f"(f[i + 8]), "+f"(f[i + 9]), "+f"(f[i + 10]), "+f"(f[i + 11]), "+f"(f[i + 12]),
                   "+f"(f[i + 13]), "+f"(f[i + 14]), "+f"(f[i + 15])
                 :
                 : "memory");
}
// What ask_sums asked for.
__device__ __forceinline__ void take_sums(float (&f)[2][32]) {
  tmem_wait_ld();
  hold32(f[0]), hold32(f[1]);
}

// The next run's sums, added to those of the runs in front: eight at a time, for want
// of registers.
__device__ __forceinline__ void add_sums(uint32_t from, float (&f)[2][32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float v[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(from + q * 8)
                 : "memory");
    tmem_wait_ld();
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                 :
                 : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) f[q >> 2][(q & 3) * 8 + j] += v[j];
  }
}

// 32 bytes, a sector, from registers.
__device__ __forceinline__ void store32(void* at, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Eight logits in units of log 2, less `base`, from the sums of words v0 .. + 7;
// `bias`: their biases in shared memory, -inf behind the vocabulary.
__device__ __forceinline__ void to_logits8(bool biased, uint32_t bias, int left, float base, float* f) {
  if (biased) {
    const float4 a = get16(bias), b = get16(bias + 16);
    f[0] = fmaf(f[0], kLog2e, a.x - base), f[1] = fmaf(f[1], kLog2e, a.y - base);
    f[2] = fmaf(f[2], kLog2e, a.z - base), f[3] = fmaf(f[3], kLog2e, a.w - base);
    f[4] = fmaf(f[4], kLog2e, b.x - base), f[5] = fmaf(f[5], kLog2e, b.y - base);
    f[6] = fmaf(f[6], kLog2e, b.z - base), f[7] = fmaf(f[7], kLog2e, b.w - base);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(f[j], kLog2e, -base);
    if (left < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = j < left ? f[j] : -INFINITY;
    }
  }
}

template <typename T, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_c, const DenseArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int S = kStages<MODE>;
  unsigned char* patches = smem + S * kStageBytes;
  unsigned char* biases = patches + kWriters * kPatchesOf<MODE> * kPatchBytes;
  DenseShared* sh = reinterpret_cast<DenseShared*>(biases + kWriters * kBiasBytes<MODE>);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kAmn = MODE >= kDw, kBmn = MODE >= kDx;

  if (MODE <= kExact && p.flags) {
    grid_wait();
    int any = 0;
    for (int m = threadIdx.x; m < p.mt; m += kThreads) any |= p.flags[m];
    if (!__syncthreads_or(any)) return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init_count(&sh->full[s], 1), mbar_init_count(&sh->empty[s], 1);
    for (int a = 0; a < 2; ++a) mbar_init_count(&sh->acc_full[a], 1), mbar_init_count(&sh->acc_empty[a], 2 * kWriters);
    sh->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWriters + 1) pair_tmem_alloc(&sh->tmem, 512);
  if (warp == kWriters && lane == 0) {
    tma_prefetch_map(&map_a), tma_prefetch_map(&map_b);
    if (MODE > kExact && p.out_cols) tma_prefetch_map(&map_c);
  }
  if (MODE != kDx || !p.beside) grid_wait();
  grid_let_next();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  const uint32_t tmem = sh->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = p.mt * p.nt * p.parts;
  const PairWait wait{&sh->stop, p.abandoned, p.wait};

  if (warp == kWriters) {
    // ---- loads
    const uint32_t base = smem_u32(smem);
    const uint32_t full0 = map_rank(smem_u32(&sh->full[0]), 0);
    const int half = p.width / 2, chunks = (half + 63) / 64;
    const uint32_t bytes = kSideBytes + (kBmn ? chunks * kChunkBytes : half * 128);
    uint32_t s = 0, phase = 1;
    bool ok = true;
    for (int idx = pair; ok && !p.stall && idx < units; idx += pairs) {
      const Unit u = unit_at<T, MODE>(p, idx);
      if (MODE <= kExact && p.flags && !p.flags[u.m0 / kTile]) continue;
      const int ma = u.m0 + (int)rank * 128, nb = u.n0 + (int)rank * half;
      for (int b = 0; b < u.blocks; ++b) {
        if (!(ok = __all_sync(~0u, pair_wait(&sh->empty[s], phase, wait)))) break;
        const uint32_t bar = full0 + s * 8, sa = base + s * kStageBytes, sb = sa + kSideBytes;
        const int d = u.d0 + b * kBlock;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_tx(&sh->full[s], 2 * bytes);  // both CTAs' bytes
          if (kAmn) {
            tma_load_2d(sa, &map_a, ma, d, bar);
            tma_load_2d(sa + kChunkBytes, &map_a, ma + 64, d, bar);
          } else {
            tma_load_2d(sa, &map_a, d, ma, bar);
          }
          if (kBmn) {
            tma_load_2d(sb, &map_b, nb, d, bar);
            if (chunks > 1) tma_load_2d(sb + kChunkBytes, &map_b, nb + 64, d, bar);
          } else {
            tma_load_2d(sb, &map_b, d, nb, bar);
          }
        }
        __syncwarp();
        if (++s == S) s = 0, phase ^= 1;
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
      const uint32_t idesc = pair_idesc(kBf16, kAmn, kBmn, p.width);
      for (int idx = pair; ok && idx < units; idx += pairs) {
        const Unit u = unit_at<T, MODE>(p, idx);
        if (MODE <= kExact && p.flags && !p.flags[u.m0 / kTile]) continue;
        const int last = (p.depth - u.d0 - (u.blocks - 1) * kBlock + 15) / 16;  // steps of the last block
        for (int r0 = 0; ok && r0 < u.blocks; r0 += u.run, ++n) {
          const uint32_t a = n & 1, d = tmem + a * kTile;
          if (!(ok = __all_sync(~0u, pair_wait(&sh->acc_empty[a], (n >> 1 & 1) ^ 1, wait)))) break;
          tc_fence_after();
          const int end = min(r0 + u.run, u.blocks);
          for (int b = r0; b < end; ++b) {
            if (!(ok = __all_sync(~0u, pair_wait(&sh->full[s], phase, wait)))) break;
            tc_fence_after();
            const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
            const int steps = b == u.blocks - 1 ? min(last, kBlock / 16) : kBlock / 16;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBlock / 16; ++k)
                if (k < steps) pair_mma(d, da + k * (kAmn ? 128 : 2), db + k * (kBmn ? 128 : 2), idesc, b > r0 || k > 0);
              pair_commit(&sh->empty[s]);
              if (b == end - 1) pair_commit(&sh->acc_full[a]);
            }
            __syncwarp();
            if (++s == S) s = 0, phase ^= 1;
          }
        }
      }
      if (!ok) {
        for (const uint64_t t0 = global_ns(); global_ns() - t0 < 20000000ull;) __nanosleep(1000);
      }
    }
  } else {
    // ---- results
    const int quarter = warp & 3, share = warp >> 2;  // TMEM lanes 32 quarter .. + 31; columns 64 share .. + 63
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t patch = smem_u32(patches + warp * kPatchesOf<MODE> * kPatchBytes);
    const uint32_t bias = smem_u32(biases + warp * kBiasBytes<MODE>);
    const int c = share * 64;
    uint32_t n = 0;
    bool lost = false;  // a wait ran out: what is left to write is NaN
    for (int idx = pair; idx < units; idx += pairs) {
      const Unit u = unit_at<T, MODE>(p, idx);
      if (MODE <= kExact && p.flags && !p.flags[u.m0 / kTile]) continue;
      const int m0 = u.m0 + (int)rank * 128 + quarter * 32, row = m0 + lane;
      const bool some = c < min(p.width, p.ndim - u.n0) && m0 < p.mdim;  // the same in all lanes
      int y = kIgnored;
      float lse = 0.f;
      if (MODE <= kExact) {
        if (row < p.mdim) {
          y = p.cols[row];
          if (MODE != kStats) lse = p.lse[row];
        }
        if (p.bias && some) {
          const float2 v = *reinterpret_cast<const float2*>(p.bias + u.n0 + c + 2 * lane);
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(bias + lane * 8), "f"(v.x), "f"(v.y) : "memory");
        }
      }
      // the warp's columns; once they are in registers the accumulator is another tile's
      float sums[2][32];
      int r0 = 0;  // the run's first block
      do {
        const uint32_t a = n & 1, from = tmem + a * kTile + lanes + c;
        if (!lost && !__all_sync(~0u, pair_wait(&sh->acc_full[a], n >> 1 & 1, wait))) {
          lost = true;
          *p.lost = 1;
        }
        tc_fence_after();
        if (some && r0 == 0) {
          ask_sums(from, sums[0]), ask_sums(from + 32, sums[1]);
          take_sums(sums);
        } else if (some) {
          add_sums(from, sums);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_rank(smem_u32(&sh->acc_empty[a]), 0));
        ++n, r0 += u.run;
      } while (MODE >= kDw && r0 < u.blocks);
      if (lost) {  // sums that never came
#pragma unroll
        for (int j = 0; j < 32; ++j) sums[0][j] = sums[1][j] = __int_as_float(0x7FC00000);
      }
      const float scale = MODE >= kDw ? *p.scale : 1.f;
      const int left = p.ndim - u.n0 - c;  // words from the first column on
      const int at_target = y - u.n0 - c;
      if constexpr (MODE == kStats) {
        float top = -INFINITY, sum = 0.f;
        if (some) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              to_logits8(p.bias, bias + (h * 32 + i) * 4, left - h * 32 - i, 0.f, sums[h] + i);
          if ((unsigned)at_target < 64u) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j == at_target) sums[j >> 5][j & 31] = -INFINITY;
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 64; ++j) top = fmaxf(top, sums[j >> 5][j & 31]);
          const float base = top == -INFINITY ? 0.f : top;  // all of them -inf: a sum of zeros
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j & 3] += ex2(sums[j >> 5][j & 31] - base);
          sum = (s[0] + s[1]) + (s[2] + s[3]);
        }
        p.top[(int64_t)(kShares * u.tile_n + share) * p.ld + row] = top;
        p.sum[(int64_t)(kShares * u.tile_n + share) * p.ld + row] = sum;
      } else if constexpr (MODE <= kExact) {
        float sum = 0.f;
        if (some) {
          const uint32_t keep = y == kIgnored ? 0u : ~0u;  // such a row may hold anything: exactly 0
          if (MODE == kFirst && (unsigned)at_target < 64u) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j == at_target) sums[j >> 5][j & 31] = -INFINITY;
          }
          __syncwarp();
          T* o = static_cast<T*>(p.out) + row * p.ldo + u.n0 + c;
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 64; i += 16) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float* f = sums[i >> 5] + (i & 31) + 8 * k;
              to_logits8(p.bias, bias + (i + 8 * k) * 4, left - i - 8 * k, lse, f);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                f[j] = MODE == kExact ? kUp<T> * ex2(f[j]) : ex2(f[j]);
                if (MODE == kFirst) s[j & 3] += f[j];
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) w[4 * k + j] = pack2<T>(f[2 * j], f[2 * j + 1]) & keep;
            }
            if (row < p.mdim) store32(o + i, w);
          }
          sum = (s[0] + s[1]) + (s[2] + s[3]);
          if (MODE == kExact && (unsigned)at_target < 64u && row < p.mdim)  // the target's probability less 1
            o[at_target] = of_f<T>(kUp<T> * expm1f(-p.losses[row]));
          __syncwarp();
        }
        if (MODE == kFirst) p.sum[(int64_t)(kShares * u.tile_n + share) * p.ld + row] = sum;
      } else if constexpr (MODE == kDw16) {
        if (some) {
          uint32_t at = patch;
          // addresses made here: held in registers beside the sums they made the compiler
          // spill (1001 rows of 5003 x 651 float16 68 us for 65)
          asm volatile("" : "+r"(at));
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float(&f)[32] = sums[h];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] *= scale;
            const int last = left - 1 - h * 32;
            if (p.db && (unsigned)last < 32u && row < p.mdim) {  // the bias's column
              float own = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == last) own = f[j];
              if (!p.db_out) p.db[row] = own;
              else if (p.db32) static_cast<float*>(p.db_out)[row] = own;
              else static_cast<T*>(p.db_out)[row] = of_f<T>(own);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put16(at + lane * 128 + (((h * 4 + i) ^ (lane & 7)) << 4), pack2<T>(f[8 * i], f[8 * i + 1]),
                    pack2<T>(f[8 * i + 2], f[8 * i + 3]), pack2<T>(f[8 * i + 4], f[8 * i + 5]),
                    pack2<T>(f[8 * i + 6], f[8 * i + 7]));
          }
          if (p.out_cols) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (m0 < p.mdim && u.n0 + c < p.out_cols) tma_store_2d(&map_c, at, u.n0 + c, m0);
              bulk_commit();
            }
          } else {  // a row of 64 values at a time, two a lane
            __syncwarp();
            const int col = u.n0 + c + 2 * lane, left = min(p.out_end, u.n0 + p.width) - col;
            T* o = static_cast<T*>(p.out) + m0 * p.ldo + col;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
              uint32_t v;
              asm volatile("ld.shared.b32 %0, [%1];"
                           : "=r"(v)
                           : "r"(at + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4)
                           : "memory");
              if (m0 + i >= p.mdim) continue;
              uint16_t* to = reinterpret_cast<uint16_t*>(o + i * p.ldo);
              if (p.even && left >= 2) {
                *reinterpret_cast<uint32_t*>(to) = v;
              } else {
                if (left >= 1) to[0] = (uint16_t)v;
                if (left >= 2) to[1] = (uint16_t)(v >> 16);
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int x = u.n0 + c + h * 32;
          if (!some || x >= min(u.n0 + p.width, p.ndim)) continue;
          const uint32_t at = patch;
          float(&f)[32] = sums[h];
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          if (MODE == kDw) {
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] *= scale;
            const int last = p.ndim - 1 - x;
            if (p.db && (unsigned)last < 32u && row < p.mdim) {  // the bias's column
              float own = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == last) own = f[j];
              float* o = p.db + u.part * p.part_rows + row;
              if (!p.db_out) *o = p.db_add ? *o + own : own;
              else if (p.db32) static_cast<float*>(p.db_out)[row] = own;
              else static_cast<T*>(p.db_out)[row] = of_f<T>(own);
            }
            if (p.out_end > p.out_cols && p.out_cols < x + 32 && row < p.mdim) {
              float* o = static_cast<float*>(p.out) + row * p.ldo + x;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (x + j >= p.out_cols && x + j < p.out_end) o[j] = p.add ? o[j] + f[j] : f[j];
            }
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            put16(at + lane * 128 + ((i ^ (lane & 7)) << 4), __float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                  __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m0 < p.mdim && x < p.out_cols) {
              const int at_row = (int)(u.part * p.part_rows) + m0;
              if (MODE == kDw && p.add) tma_add_2d(&map_c, at, x, at_row);
              else tma_store_2d(&map_c, at, x, at_row);
            }
            bulk_commit();
          }
        }
      }
    }
    if (MODE > kExact && lane == 0) bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kWriters + 1) pair_tmem_free(tmem, 512);
  if (MODE == kDx && p.beside) grid_wait();
}

// --------------------------------------------------------- around the products --

// What the kernels of a call share: made by begin_kernel.
struct Head {
  float scale;     // gradient of a loss of weight 1
  float scale_up;  // the same for sums of d * kUp
  float most;      // largest magnitude of the rows' weights
  int count;       // rows with a target
  int lost;        // a wait ran out
  int arrived;     // CTAs of the last rows_kernel
};

struct BeginArgs {
  const void* target;
  int wide;  // int64 targets
  int64_t rows, ignore;
  int vocab, padded;  // values of `bias2`
  const void* bias;
  float* bias2;
  int32_t* cols;
  const float* row_scale;
  const float* scale_dev;
  float scale, up;
  int mean;
  Head* head;
  float* ref;          // the targets' logits, in units of log 2
  int* flags;          // of every 256 rows: cleared; nullptr: none
  const void *x, *w;
  int64_t ldx, ldw;
  int width;
};

// x . w by a warp.
template <typename T>
__device__ __forceinline__ float dot_of(const T* x, const T* w, int width) {
  const int lane = threadIdx.x & 31;
  float sum = 0.f;
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15) == 0) {
    done = width & ~7;
    for (int c = lane * 8; c < done; c += 256) {
      alignas(16) T a[8], b[8];
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(x + c);
      *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(w + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(to_f(a[j]), to_f(b[j]), sum);
    }
  }
#pragma unroll 8
  for (int c = done + lane; c < width; c += 32) sum = fmaf(to_f(x[c]), to_f(w[c]), sum);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}

__device__ __forceinline__ int column_of(const BeginArgs& p, int64_t t) {
  const int64_t y = p.wide ? static_cast<const int64_t*>(p.target)[t] : static_cast<const int32_t*>(p.target)[t];
  return y == p.ignore ? kIgnored : y >= 0 && y < p.vocab ? (int)y : kOutside;
}

// Columns and logits of the targets (the latter as float32 sums: float16 products
// are cut by the tensor cores, see psgd_experts.cu, and this logit counts most),
// the bias in units of log 2, and (first CTA) what the gradients are scaled by.
template <typename T, typename B>
__global__ void __launch_bounds__(1024) begin_kernel(const BeginArgs p) {
  grid_wait();
  grid_let_next();
  const int64_t first = (int64_t)blockIdx.x * 1024 + threadIdx.x, step = (int64_t)gridDim.x * 1024;
  if (p.bias)
    for (int64_t v = first; v < p.padded; v += step)
      p.bias2[v] = v < p.vocab ? to_f(static_cast<const B*>(p.bias)[v]) * kLog2e : -INFINITY;
  if (p.flags)
    for (int64_t m = first; m * kTile < p.rows; m += step) p.flags[m] = 0;
  for (int64_t t = first >> 5; t < p.rows; t += step >> 5) {
    const int y = column_of(p, t);
    float v = 0.f;
    if (y >= 0) {
      v = dot_of(static_cast<const T*>(p.x) + t * p.ldx, static_cast<const T*>(p.w) + y * p.ldw, p.width) * kLog2e;
      if (p.bias) v = fmaf(to_f(static_cast<const B*>(p.bias)[y]), kLog2e, v);
    }
    if ((threadIdx.x & 31) == 0) p.ref[t] = v, p.cols[t] = y;
  }
  if (blockIdx.x) return;
  __shared__ int s_count[32];
  __shared__ float s_most[32];
  int count = 0;
  float most = 0.f;
  for (int64_t t = threadIdx.x; t < p.rows; t += 1024) {
    if (column_of(p, t) == kIgnored) continue;
    ++count;
    if (p.row_scale) most = fmaxf(most, fabsf(p.row_scale[t]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    count += __shfl_xor_sync(~0u, count, o);
    most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
  }
  if ((threadIdx.x & 31) == 0) s_count[threadIdx.x >> 5] = count, s_most[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) count += s_count[w], most = fmaxf(most, s_most[w]);
    float scale = p.scale_dev ? p.scale * *p.scale_dev : p.scale;
    if (p.mean) scale = count ? scale / (float)count : 0.f;
    if (p.row_scale) scale *= most;
    *p.head = Head{scale, scale / p.up, most, count, 0, 0};
  }
}

// The loss of a row from its largest logit but the target's, the others' sum of
// exponentials beside that, and the target's logit (in units of log 2).
__device__ __forceinline__ float loss_from(float top, float sum, float mine) {
  if (mine == INFINITY) return mine - mine;  // NaN: infinity less infinity is not 0
  const float base = top == -INFINITY ? 0.f : top, over = base - mine;
  return sum == 0.f    ? mine - mine
         : over < 64.f ? log1pf(sum * exp2f(over))
                       : (over + log2f(sum + exp2f(-over))) * kLn2;
}

// The logarithm of the sum of all of a row's exponentials, from the same.  The larger
// of the two parts stays in front: taken from the loss (lse = loss + mine) it would
// cancel where the target is far below the others, to nothing at a mask of -1e9.
__device__ __forceinline__ float lse_from(float top, float sum, float mine) {
  const float over = mine - top;
  return sum == 0.f   ? mine
         : over > 0.f ? mine + log2f(fmaf(sum, exp2f(-over), 1.f))
                      : top + log2f(sum + exp2f(over));
}

struct RowsArgs {
  const float *top, *sum, *mine;  // [tile's share][ld], and the targets' logits
  int tiles, ld;                  // shares of tiles
  const int32_t* cols;
  int rows;
  float* losses;
  // gradients
  float *lse, *factor;     // log2 of the sum of exponentials; the row's weight in units of the largest; nullptr: no gradients
  const float* row_scale;
  const void* x;           // rows on 16-byte boundaries
  int64_t ldx;
  void* xs;                // x times the row's factor, then (with a bias) the factor itself
  int64_t ldxs;
  int width, bias;         // values of x that it takes
  const Head* head;
  // after the first product alone: the exponentials'
  // buffer gets the targets' values; a row whose sum is out of range flags its 256
  void* e;
  int64_t lde;
  int* set;
  const int* flags;  // 256 rows that are taken; nullptr: all
  // the reduced loss of all rows, by the CTA that ends last; nullptr: not here
  float* loss;
  const float* all_losses;
  int64_t all_rows;
  int mean;
  int* arrived;
};
constexpr float kMostSum = 1.8446744e19f;  // 2^64

constexpr int kRowsOfCta = 8, kRowGroups = 32, kRowsThreads = kRowsOfCta * kRowGroups;

// A chunk's statistics, put together from the tiles': eight rows a CTA, the tiles
// shared by 32 threads a row.
template <typename T>
__device__ __forceinline__ void rows_of_cta(const RowsArgs& p) {
  __shared__ float s_top[kRowGroups][kRowsOfCta], s_sum[kRowGroups][kRowsOfCta], s_factor[kRowsOfCta];
  const int r = threadIdx.x % kRowsOfCta, g = threadIdx.x / kRowsOfCta, t = blockIdx.x * kRowsOfCta + r;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 8
  for (int n = g; n < p.tiles; n += kRowGroups) {
    const float b = p.sum[(int64_t)n * p.ld + t];
    if (p.e) {
      sum += b;
      continue;
    }
    const float a = p.top[(int64_t)n * p.ld + t];
    const float high = fmaxf(top, a), base = high == -INFINITY ? 0.f : high;
    sum = sum * ex2(top - base) + b * ex2(a - base);
    top = high;
  }
  s_top[g][r] = p.e ? 0.f : top, s_sum[g][r] = sum;
  __syncthreads();
  if (g == 0) {
    float high = s_top[0][r];
#pragma unroll
    for (int i = 1; i < kRowGroups; ++i) high = fmaxf(high, s_top[i][r]);
    const float base = high == -INFINITY ? 0.f : high;
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kRowGroups; ++i) all += s_sum[i][r] * ex2(s_top[i][r] - base);
    float factor = 0.f;
    if (t < p.rows) {
      const int y = p.cols[t];
      const float nan = __int_as_float(0x7FC00000);
      float loss = 0.f, lse = 0.f;
      if (y >= 0) {
        const float mine = p.mine[t];
        if (mine == INFINITY) all = nan;  // and so are its gradients, though the exponentials beside it are 0
        loss = p.e ? log1pf(all) : loss_from(high, all, mine);
        if (!p.e) lse = lse_from(high, all, mine);
        factor = p.row_scale ? (p.head->most > 0.f ? p.row_scale[t] / p.head->most : p.row_scale[t]) : 1.f;
        if (p.e) {
          // the buffer holds exp(l - mine): d is that times the target's
          // probability, and the target's own d the rest's sum, negative
          if (!(all < kMostSum)) p.set[t / kTile] = 1;
          factor /= 1.f + all;
          static_cast<T*>(p.e)[t * p.lde + y] = of_f<T>(-all);
        }
      }
      if (y == kOutside || p.head->lost) loss = lse = factor = nan;
      p.losses[t] = loss;
      if (p.factor) {
        if (!p.e) p.lse[t] = lse;
        p.factor[t] = factor;
      }
    }
    s_factor[r] = factor;
  }
  if (!p.factor) return;
  __syncthreads();
  const int vecs = (int)(p.ldxs / 8), r0 = blockIdx.x * kRowsOfCta;
  for (int i = threadIdx.x; i < kRowsOfCta * vecs; i += kRowsThreads) {
    const int q = i / vecs, c = (i - q * vecs) * 8, row = r0 + q;
    if (row >= p.rows) break;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx + c;
    const float f = s_factor[q];
    alignas(16) T v[8];
    if (c + 8 <= p.width) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < p.width ? x[j] : of_f<T>(c + j == p.width && p.bias ? 1.f : 0.f);
    }
    if (f == 0.f) {  // whatever the row holds
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = of_f<T>(0.f);
    } else if (f != 1.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = of_f<T>(to_f(v[j]) * f);
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(p.xs) + row * p.ldxs + c) = *reinterpret_cast<const uint4*>(v);
  }
}

// The sum of every loss, or their mean, by one CTA in a fixed order.
template <int THREADS>
__device__ __forceinline__ void reduce_losses(const float* losses, int64_t rows, int mean, const Head* head, float* loss) {
  __shared__ double s_sum[32];
  double sum = 0.0;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < rows; t += THREADS) sum += (double)__ldcg(losses + t);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < THREADS / 32; ++w) sum += s_sum[w];
  // 0 / 0 where every row is ignored
  *loss = head->lost ? __int_as_float(0x7FC00000) : (float)(mean ? sum / (double)head->count : sum);
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsArgs p) {
  grid_wait();
  grid_let_next();
  if (!p.flags || p.flags[blockIdx.x * kRowsOfCta / kTile]) rows_of_cta<T>(p);
  if (!p.loss) return;
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(p.arrived, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  reduce_losses<kRowsThreads>(p.all_losses, p.all_rows, p.mean, p.head, p.loss);
}

// ----------------------------------------------------------------- one row --
//
// The loss of one row without gradients: each word's values are read once, as they
// lie, by a warp, kWords words at a time; the row is in shared memory.  Bound by
// reading the matrix: 33278 x 650 bfloat16 14.6 us (3.0 TB/s) and 4 for the end,
// where the products, which copy such rows first, take 41.  (The same for eight
// rows: 49, the products 38.)
constexpr int kWords = 4, kOneThreads = 256;
constexpr int kOneBytes = 44 << 10;  // of the row, in float32

struct OneArgs {
  const void *x, *w, *bias, *target;
  int64_t ldw, ignore;
  int wide, vocab, width;
  float *top, *sum, *mine;  // of each CTA, and the target's logit
  int parts;
  float *losses, *loss;     // either may be nullptr
  bool ignored_nan;         // of a mean
};

__device__ __forceinline__ int column_of(const OneArgs& p) {
  const int64_t y = p.wide ? *static_cast<const int64_t*>(p.target) : *static_cast<const int32_t*>(p.target);
  return y == p.ignore ? kIgnored : y >= 0 && y < p.vocab ? (int)y : kOutside;
}

// The products of VEC values of a few words with the row's.
template <typename T, int VEC>
__device__ __forceinline__ void add_words(float (&acc)[kWords], const T (&a)[kWords][VEC], const float* x) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float v = x[j];
#pragma unroll
    for (int q = 0; q < kWords; ++q) acc[q] = fmaf(to_f(a[q][j]), v, acc[q]);
  }
}

// VEC values of a word at a time: 8 where rows start on 16-byte boundaries, 2 on
// 4-byte ones.
template <typename T, typename B, int VEC>
__global__ void __launch_bounds__(kOneThreads) one_kernel(const OneArgs p) {
  extern __shared__ float smem[];
  __shared__ float s_top[kOneThreads / 32], s_sum[kOneThreads / 32];
  // steps in flight, 512 or 320 values a word: timed at a width of 650 alone.  What they
  // leave of a row (10 values of 650, 448 of 960) is read value by value.
  constexpr int U = VEC == 8 ? 2 : 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, step = 32 * VEC;
  const int pitch = (p.width + step - 1) / step * step;
  grid_wait();
  grid_let_next();
  for (int c = threadIdx.x; c < pitch; c += kOneThreads) smem[c] = c < p.width ? to_f(static_cast<const T*>(p.x)[c]) : 0.f;
  const int y = column_of(p);
  float top = -INFINITY, sum = 0.f;
  __syncthreads();
  const int stride = (int)gridDim.x * (kOneThreads / 32) * kWords;
  for (int v0 = ((int)blockIdx.x * (kOneThreads / 32) + warp) * kWords; v0 < p.vocab; v0 += stride) {
    float acc[kWords];
#pragma unroll
    for (int q = 0; q < kWords; ++q) acc[q] = 0.f;
    const T* w = static_cast<const T*>(p.w) + (int64_t)v0 * p.ldw;
    const int words = min(kWords, p.vocab - v0);
    // several steps' loads in flight, then the rest one by one
    int c0 = 0;
    for (; c0 + U * step <= p.width; c0 += U * step) {
      alignas(16) T a[U][kWords][VEC];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          const T* at = w + (q < words ? q : 0) * p.ldw + c0 + i * step + lane * VEC;
          if constexpr (VEC == 8) *reinterpret_cast<uint4*>(a[i][q]) = __ldcs(reinterpret_cast<const uint4*>(at));
          else if constexpr (VEC == 2) *reinterpret_cast<uint32_t*>(a[i][q]) = __ldcs(reinterpret_cast<const uint32_t*>(at));
          else a[i][q][0] = at[0];
        }
#pragma unroll
      for (int i = 0; i < U; ++i) add_words<T, VEC>(acc, a[i], smem + c0 + i * step + lane * VEC);
    }
    for (int c = c0 + lane * VEC; c < p.width; c += step) {
      alignas(16) T a[kWords][VEC];
#pragma unroll
      for (int q = 0; q < kWords; ++q)
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[q][j] = c + j < p.width ? w[(q < words ? q : 0) * p.ldw + c + j] : of_f<T>(0.f);
      add_words<T, VEC>(acc, a, smem + c);
    }
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      const float b = p.bias && q < words ? to_f(static_cast<const B*>(p.bias)[v0 + q]) * kLog2e : 0.f;
      float l = acc[q];
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      l = fmaf(l, kLog2e, b);
      if (q >= words) continue;
      if (v0 + q == y) {
        if (lane == 0) *p.mine = l;
        continue;
      }
      const float high = fmaxf(top, l), base = high == -INFINITY ? 0.f : high;
      sum = sum * ex2(top - base) + ex2(l - base);
      top = high;
    }
  }
  if (lane == 0) s_top[warp] = top, s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  float high = -INFINITY, all = 0.f;
  for (int i = 0; i < kOneThreads / 32; ++i) high = fmaxf(high, s_top[i]);
  const float base = high == -INFINITY ? 0.f : high;
  for (int i = 0; i < kOneThreads / 32; ++i) all += s_sum[i] * ex2(s_top[i] - base);
  p.top[blockIdx.x] = high, p.sum[blockIdx.x] = all;
}

// The CTAs' statistics put together by a warp.
__global__ void __launch_bounds__(32) one_end_kernel(const OneArgs p) {
  grid_wait();
  const int lane = threadIdx.x;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 8
  for (int i = lane; i < p.parts; i += 32) {
    const float a = p.top[i], b = p.sum[i];
    const float high = fmaxf(top, a), base = high == -INFINITY ? 0.f : high;
    sum = sum * ex2(top - base) + b * ex2(a - base);
    top = high;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float a = __shfl_xor_sync(~0u, top, o), b = __shfl_xor_sync(~0u, sum, o);
    const float high = fmaxf(top, a), base = high == -INFINITY ? 0.f : high;
    sum = sum * ex2(top - base) + b * ex2(a - base);
    top = high;
  }
  if (lane) return;
  const int y = column_of(p);
  const float nan = __int_as_float(0x7FC00000);
  const float loss = y == kIgnored ? 0.f : y == kOutside ? nan : loss_from(top, sum, *p.mine);
  if (p.losses) *p.losses = loss;
  if (p.loss) *p.loss = loss;
  if (p.loss && p.ignored_nan && y == kIgnored) *p.loss = nan;  // the mean of nothing
}

struct JoinArgs {
  const float* part;
  int64_t step;  // between parts
  int parts;
  int64_t rows, ldp;
  int cols;
  void* out;
  int64_t ldo;
  bool aligned, add;
  const float* factor;  // of each row, times head->scale_up; nullptr: none
  const Head* head;
  // the reduced loss, by the first CTA; nullptr: not here
  float* loss;
  const float* losses;
  int64_t all_rows;
  int mean;
};

// out = the sum of a product's parts, four values a thread and step.
template <typename O>
__global__ void __launch_bounds__(256) join_kernel(const JoinArgs p) {
  grid_wait();
  grid_let_next();
  if (p.loss && blockIdx.x == 0) reduce_losses<256>(p.losses, p.all_rows, p.mean, p.head, p.loss);
  const int vecs = (int)(p.ldp / 4);
  const int64_t n = p.rows * vecs;
  const float scale = p.factor ? p.head->scale_up : 1.f;
  const bool lost = p.head->lost;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = n < ((int64_t)1 << 32) ? (uint32_t)i / (uint32_t)vecs : i / vecs;
    const int c = (int)(i - row * vecs) * 4;
    const float* at = p.part + row * p.ldp + c;
    float4 s = *reinterpret_cast<const float4*>(at);
    for (int k = 1; k < p.parts; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(at + k * p.step);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    float v[4] = {s.x, s.y, s.z, s.w};
    if (p.factor) {
      const float f = p.factor[row] * scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f == 0.f ? 0.f : v[j] * f;
    }
    O* o = static_cast<O*>(p.out) + row * p.ldo + c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (lost) v[j] = __int_as_float(0x7FC00000);
      if (p.add && c + j < p.cols) v[j] += to_f(o[j]);
    }
    if (p.aligned && c + 4 <= p.cols) {
      if constexpr (sizeof(O) == 4) *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      else *reinterpret_cast<uint2*>(o) = make_uint2(pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < p.cols) o[j] = of_f<O>(v[j]);
    }
  }
}

// The bias's gradient from its sums, and the reduced loss.
struct EndArgs {
  const float* losses;
  int64_t rows;
  float* loss;  // nullptr: not wanted
  int mean;
  const float* sums;  // of the bias's gradient, `parts` of them `step` apart
  int64_t step;
  int parts, vocab;
  void* db;  // nullptr: none
  bool add;
  const Head* head;
};

template <typename B>
__global__ void __launch_bounds__(1024) end_kernel(const EndArgs p) {
  grid_wait();
  const float nan = __int_as_float(0x7FC00000);
  const bool lost = p.head->lost;
  if (p.db)
    for (int64_t v = (int64_t)blockIdx.x * 1024 + threadIdx.x; v < p.vocab; v += (int64_t)gridDim.x * 1024) {
      float s = p.sums[v];
      for (int k = 1; k < p.parts; ++k) s += p.sums[k * p.step + v];
      B* o = static_cast<B*>(p.db) + v;
      if (p.add) s += to_f(*o);
      *o = of_f<B>(lost ? nan : s);
    }
  if (blockIdx.x == 0 && p.loss) reduce_losses<1024>(p.losses, p.rows, p.mean, p.head, p.loss);
}

// ------------------------------------------------------------------- host --

using Args = psgd_cross_entropy_args;

constexpr int kPairs = 76;
constexpr int64_t kOneCtas = 152 * 4;  // of one_kernel
// Products of fewer multiplications compute the logits twice: of 8192 or 16384
// words of 512 values, 512 rows took 53 and 67 us so, 59 and 59 with one product.
constexpr double kFirstWork = 3e9;
// Bytes of a chunk's buffers, about: a chunk more reads and writes dW's float32 sums
// once more, which of 16384 rows of 65536 x 2048 (2.4 GB of buffers) takes 7.08 ms in
// one chunk, 7.65 in two, 7.76 in three.
constexpr int64_t kChunk = (int64_t)1 << 32;
// Rows that a product over them sums in one go, 64 runs at most.
constexpr int64_t kMostRows = 65536;

int64_t up(int64_t v, int64_t to) { return ceil_div(v, to) * to; }

// How a call is cut, and where its workspace holds what.
struct Plan {
  bool grads, dx, dw, db;
  bool one;              // no products: one row, by one_kernel
  bool direct, half;     // dw: the product writes it, in float32 or 16 bits
  bool db_now;           // db: the product writes it
  bool rows16;           // dw in 16 bits: TMA writes it
  bool first;            // one product for statistics and exponentials
  int64_t rows, chunks;  // of a chunk (a multiple of 256, but for a single one)
  int64_t lde, ldxs, ldp, ldw;
  int64_t cols_x;        // columns of x that the product over the rows takes: none for db alone
  int wide;              // words of a tile of the logits
  int nx, nw;            // columns of a tile of dx and dw
  int px, pw;            // parts of their contractions
  // offsets in the workspace
  size_t copies, cols, bias, head, losses, top, sum, mine, lse, ref, flags, factor, xs, e, part, sums, db_sums, bytes;
};

// Columns of a tile: n values in equal tiles, a multiple of `to`.
int equal_tiles(int64_t n, int to) { return (int)up(ceil_div(n, ceil_div(n, kTile)), to); }

// Words of a tile: 256, or fewer where that fills the last wave of tiles better
// (a stage of a tile costs 150 ns and 0.7 ns a column).  64 rows of 1000 x 4096 with
// gradients: 78 us with 256, 69 so.
int logits_tile(int64_t mt, int64_t vocab) {
  int best = kTile;
  double least = 0;
  for (int w = kTile; w >= 64; w -= 64) {
    const double cost = (double)ceil_div(mt * ceil_div(vocab, w), kPairs) * (150.0 + 0.7 * w);
    if (w == kTile || cost < least) least = w == kTile ? 0.97 * cost : cost, best = w;
  }
  return best;
}

// Parts of a contraction of `blocks`: what fills the last wave best, given that
// a block of a tile takes 0.35 us and a part of the sums `part_us`.  2240 rows of
// 33278 x 650: 326 us with one part of each, 265 so; 1024 of 8192 x 2048 118, 108.
int parts_of(int64_t tiles, int64_t blocks, double part_us, int64_t least) {
  int best = 1;
  double time = 0;
  for (int p = 1; p <= 16 && p <= blocks; ++p) {
    const double t = (double)ceil_div(tiles * p, kPairs) * (0.35 * (double)ceil_div(blocks, p) + 1.5) + p * part_us;
    if (p == 1 || t < 0.98 * time) time = t, best = p;
  }
  return (int)std::min<int64_t>(blocks, std::max<int64_t>(best, least));
}

Operand operand_x(const Args& a) { return Operand{a.x, a.ldx, 0, 1, a.rows, a.width}; }
Operand operand_w(const Args& a) { return Operand{a.w, a.ldw, 0, 1, a.vocab, a.width}; }

Plan plan_of(const Args& a) {
  Plan p = {};
  p.dx = a.dx, p.dw = a.dw, p.db = a.db;
  p.grads = p.dx || p.dw || p.db;
  const int64_t H = a.width, V = a.vocab;
  p.cols_x = p.dw ? H : 0;
  const int64_t K = std::max<int64_t>(p.cols_x + p.db, 1);  // columns of the product over the rows
  p.lde = up(V, 64), p.ldxs = up(p.cols_x + p.db, 8), p.ldp = up(H, 4), p.ldw = up(H, 4);
  const int64_t row = p.grads ? 2 * p.lde + 2 * p.ldxs + 8 * p.ldp : 8 * kShares * ceil_div(V, kTile);
  int64_t most = std::max<int64_t>(kTile, kChunk / row / kTile * kTile);
  if (p.dw || p.db) most = std::min(most, kMostRows);
  p.chunks = std::max<int64_t>(1, ceil_div(a.rows, most));
  p.rows = p.chunks == 1 ? a.rows : up(ceil_div(a.rows, p.chunks), kTile);
  if (p.rows) p.chunks = ceil_div(a.rows, p.rows);
  const int64_t padded = up(p.rows, kTile), mt = padded / kTile;
  p.wide = logits_tile(mt, V);
  p.nx = equal_tiles(H, 32), p.nw = equal_tiles(K, 32);
  const int64_t vb = ceil_div(V, kBlock), tb = std::max<int64_t>(1, ceil_div(p.rows, kBlock));
  const int64_t most_blocks = a.dtype == PSGD_F16 ? 512 : 4096;  // what the tensor cores' truncation allows
  p.px = parts_of(mt * ceil_div(H, p.nx), vb, (double)padded * p.ldp * 8 / 4e6, ceil_div(vb, most_blocks));
  p.pw = parts_of(ceil_div(V, kTile) * ceil_div(K, p.nw), tb, (double)V * up(p.cols_x, 4) * 8 / 4e6, 1);
  p.first = p.grads && a.dtype == PSGD_BF16 && (double)a.rows * (double)V * (double)H > kFirstWork;
  p.direct = p.dw && a.dw_dtype == PSGD_F32 && reinterpret_cast<uintptr_t>(a.dw) % 16 == 0 && a.lddw % 4 == 0;
  // 16 bits: where there is nothing to add to, and enough tiles to leave them whole
  const int64_t tiles_w = ceil_div(V, kTile) * ceil_div(K, p.nw);
  p.half = p.dw && a.dw_dtype != PSGD_F32 && p.chunks == 1 && !a.accumulate && (p.pw == 1 || tiles_w >= kPairs);
  p.rows16 = reinterpret_cast<uintptr_t>(a.dw) % 16 == 0 && a.lddw % 8 == 0 && H % 8 == 0;
  if (p.half && p.rows16) p.nw = equal_tiles(K, 64);  // TMA takes patches of 64 columns
  if (p.direct || p.half) p.pw = 1;
  p.db_now = p.db && p.pw == 1 && p.chunks == 1 && !a.accumulate;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 1023) / 1024 * 1024;
    return here;
  };
  p.one = !p.grads && a.rows == 1 && up(H, 256) * 4 <= kOneBytes;
  if (p.one) {
    p.top = take(kOneCtas * 4), p.sum = take(kOneCtas * 4), p.ref = take(4);
    p.bytes = at;
    return p;
  }
  const Operand x = operand_x(a), w = operand_w(a);
  p.copies = take(copy_bytes(x) + copy_bytes(w));
  p.cols = take(a.rows * 4);
  p.bias = take(a.bias ? (up(V, p.wide) + 32) * 4 : 0);
  p.head = take(sizeof(Head));
  p.losses = take(a.losses ? 0 : a.rows * 4);
  p.top = take(kShares * ceil_div(V, p.wide) * padded * 4);
  p.sum = take(kShares * ceil_div(V, p.wide) * padded * 4);
  p.ref = take(a.rows * 4);
  if (p.first) p.flags = take(ceil_div(a.rows, kTile) * 4);
  if (p.grads) {
    p.lse = take(padded * 4);
    p.factor = take(padded * 4);
    p.xs = take(p.rows * p.ldxs * 2);
    p.e = take(p.rows * p.lde * 2);
    if (p.dx) p.part = take((size_t)p.px * padded * p.ldp * 4);
    const int64_t vp = up(V, kTile);
    if (p.db) p.db_sums = take((size_t)p.pw * vp * 4);
    if (p.dw && !p.direct && !p.half) p.sums = take((size_t)p.pw * vp * p.ldw * 4);
  }
  p.bytes = at;
  return p;
}

int sms_of(int dev, int* sms) {
  CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return PSGD_OK;
}

struct Call {
  int dev, sms;
  unsigned* abandoned;
  cudaStream_t stream;
};

template <typename T, int MODE>
int dense(const Call& c, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d, DenseArgs p) {
  static thread_local uint64_t ready = 0;
  const auto kernel = dense_kernel<T, MODE>;
  const int rc = allow_smem(kernel, dense_smem<MODE>(), c.dev, &ready);
  if (rc) return rc;
  p.mt = (int)ceil_div(p.mdim, kTile), p.nt = (int)ceil_div(p.ndim, p.width);
  if (!p.parts) p.parts = 1;
  p.stall = wait_stalls(), p.wait = wait_limit(), p.abandoned = c.abandoned;
  const int64_t pairs = std::min<int64_t>(c.sms / 2, (int64_t)p.mt * p.nt * p.parts);
  return launch_behind(kernel, dim3((unsigned)(2 * pairs)), kThreads, dense_smem<MODE>(), c.stream, a, b, d, p);
}

template <typename T, typename B>
int one_of(const Args& a, const Plan& p, unsigned char* ws, cudaStream_t stream) {
  OneArgs f = {};
  f.x = a.x, f.w = a.w, f.bias = a.bias, f.target = a.target, f.ldw = a.ldw, f.ignore = a.ignore_index;
  f.wide = a.target_bytes == 8, f.vocab = (int)a.vocab, f.width = (int)a.width;
  f.top = reinterpret_cast<float*>(ws + p.top), f.sum = reinterpret_cast<float*>(ws + p.sum);
  f.mine = reinterpret_cast<float*>(ws + p.ref);
  f.losses = a.losses, f.loss = a.loss, f.ignored_nan = a.mean;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.w) | (uintptr_t)(a.vocab > 1 ? a.ldw * 2 : 0);
  const int vec = at % 16 == 0 ? 8 : at % 4 == 0 ? 2 : 1;
  const size_t smem = up(a.width, 32 * vec) * 4;
  f.parts = (int)std::min<int64_t>(kOneCtas, ceil_div(a.vocab, kOneThreads / 32 * kWords));
  const dim3 grid((unsigned)f.parts);
  const int rc = vec == 8   ? launch_behind(one_kernel<T, B, 8>, grid, kOneThreads, smem, stream, f)
                 : vec == 2 ? launch_behind(one_kernel<T, B, 2>, grid, kOneThreads, smem, stream, f)
                            : launch_behind(one_kernel<T, B, 1>, grid, kOneThreads, smem, stream, f);
  return rc ? rc : launch_behind(one_end_kernel, dim3(1), 32, 0, stream, f);
}

template <typename T, typename B>
int loss_of(const Args& a, const Plan& p, unsigned char* ws, cudaStream_t stream) {
  Call call{};
  call.stream = stream;
  int rc;
  CUDA_TRY(cudaGetDevice(&call.dev));
  if ((rc = sms_of(call.dev, &call.sms)) || (rc = abandoned_of(call.dev, &call.abandoned)) ||
      (rc = report_abandoned(call.dev, call.abandoned, stream, false)))
    return rc;
  if (p.one) return one_of<T, B>(a, p, ws, stream);
  const int dtype = a.dtype;
  Operand x = operand_x(a), w = operand_w(a);
  Head* head = reinterpret_cast<Head*>(ws + p.head);
  int32_t* cols = reinterpret_cast<int32_t*>(ws + p.cols);
  float* bias2 = a.bias ? reinterpret_cast<float*>(ws + p.bias) : nullptr;
  float* losses = a.losses ? a.losses : reinterpret_cast<float*>(ws + p.losses);
  const float upf = kUp<T>;
  BeginArgs b = {};
  b.target = a.target, b.wide = a.target_bytes == 8, b.rows = a.rows, b.ignore = a.ignore_index, b.vocab = (int)a.vocab;
  b.padded = (int)(up(a.vocab, p.wide) + 32);
  b.bias = a.bias, b.bias2 = bias2, b.cols = cols, b.row_scale = a.row_scale, b.scale_dev = a.scale_dev, b.scale = a.scale;
  b.up = upf, b.mean = a.mean, b.head = head;
  float* ref = reinterpret_cast<float*>(ws + p.ref);
  int* flags = p.first ? reinterpret_cast<int*>(ws + p.flags) : nullptr;
  b.ref = ref, b.flags = flags, b.x = x.p, b.w = w.p, b.width = (int)a.width;
  b.ldx = x.ld, b.ldw = w.ld;
  const int64_t most = std::max<int64_t>(a.rows * 32, a.bias ? a.vocab : 0);
  const unsigned ctas = (unsigned)std::max<int64_t>(1, std::min<int64_t>(call.sms * 2, ceil_div(most, 1024)));
  if ((rc = launch_behind(begin_kernel<T, B>, dim3(ctas), 1024, 0, stream, b))) return rc;
  // the copies read what begin_kernel reads, and start once it is past its own wait
  if (a.rows && (rc = make_readable(&x, &w, nullptr, ws + p.copies, stream, true))) return rc;
  const int64_t H = a.width, V = a.vocab, vp = up(V, kTile);
  for (int64_t t0 = 0; t0 < a.rows; t0 += p.rows) {
    const int64_t rows = std::min(p.rows, a.rows - t0), padded = up(rows, kTile);
    const T* xr = static_cast<const T*>(x.p) + t0 * x.ld;
    CUtensorMap mx, mw, none = {};
    const int64_t sx[2] = {H, rows}, sw[2] = {H, V}, lx = tma_stride(x.ld, H, rows), lw = tma_stride(w.ld, H, V);
    if ((rc = encode(&mx, dtype, xr, 2, sx, &lx, 128)) || (rc = encode(&mw, dtype, w.p, 2, sw, &lw, p.wide / 2))) return rc;
    DenseArgs d = {};
    d.mdim = (int)rows, d.ndim = (int)V, d.depth = (int)H, d.width = p.wide;
    d.cols = cols + t0, d.bias = bias2, d.ld = (int)padded;
    d.top = reinterpret_cast<float*>(ws + p.top), d.sum = reinterpret_cast<float*>(ws + p.sum);
    d.losses = losses + t0, d.lse = reinterpret_cast<float*>(ws + p.lse);
    d.lost = &head->lost;
    T* e = reinterpret_cast<T*>(ws + p.e);
    const int64_t se[2] = {V, rows};
    d.out = e, d.ldo = p.lde;
    RowsArgs r = {};
    r.top = d.top, r.sum = d.sum, r.mine = ref + t0, r.tiles = kShares * (int)ceil_div(V, p.wide), r.ld = (int)padded;
    r.cols = d.cols, r.rows = (int)rows, r.losses = losses + t0, r.row_scale = a.row_scale ? a.row_scale + t0 : nullptr;
    r.head = head;
    T* xs = reinterpret_cast<T*>(ws + p.xs);
    float* factor = reinterpret_cast<float*>(ws + p.factor);
    if (p.grads) {
      r.lse = reinterpret_cast<float*>(ws + p.lse), r.factor = factor;
      r.x = xr, r.ldx = lx, r.xs = xs, r.ldxs = p.ldxs, r.width = (int)p.cols_x, r.bias = p.db;
    }
    const dim3 row_ctas((unsigned)ceil_div(rows, kRowsOfCta));
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      if (p.first) {
        DenseArgs q = d;
        q.lse = r.mine;
        if ((rc = dense<T, kFirst>(call, mx, mw, none, q))) return rc;
        RowsArgs o = r;
        o.e = e, o.lde = p.lde, o.set = flags + t0 / kTile;
        if ((rc = launch_behind(rows_kernel<T>, row_ctas, kRowsThreads, 0, stream, o))) return rc;
        // what follows is for the rows that it flagged, as a rule none
        d.flags = r.flags = o.set;
      }
    }
    const bool last = t0 + p.rows >= a.rows;
    if (a.loss && last && !p.dx) {
      r.loss = a.loss, r.all_losses = losses, r.all_rows = a.rows, r.mean = a.mean, r.arrived = &head->arrived;
    }
    if ((rc = dense<T, kStats>(call, mx, mw, none, d)) ||
        (rc = launch_behind(rows_kernel<T>, row_ctas, kRowsThreads, 0, stream, r)))
      return rc;
    if (!p.grads) continue;
    if ((rc = dense<T, kExact>(call, mx, mw, none, d))) return rc;
    if (p.dw || p.db) {
      CUtensorMap ma, mb, mc = {};
      const bool own = p.direct || p.half;
      void* sums = own ? a.dw : ws + p.sums;
      const int64_t ldc = own ? tma_stride(a.lddw, H, V) : p.ldw;
      // the columns that TMA writes: whole 16 bytes of rows that start on such boundaries
      const int64_t whole = p.direct ? H / 4 * 4 : !p.dw || (p.half && !p.rows16) ? 0 : H;
      const int64_t sx2[2] = {p.cols_x + p.db, rows}, sc[2] = {std::max<int64_t>(whole, 4), own ? V : p.pw * vp};
      if ((rc = encode(&ma, dtype, e, 2, se, &p.lde, 64)) || (rc = encode(&mb, dtype, xs, 2, sx2, &p.ldxs, 64)) ||
          (whole && (rc = encode(&mc, p.half ? dtype : PSGD_F32, sums, 2, sc, &ldc, 32))))
        return rc;
      DenseArgs q = {};
      q.mdim = (int)V, q.ndim = (int)(p.cols_x + p.db), q.depth = (int)rows, q.width = p.nw;
      q.parts = (int)std::min<int64_t>(p.pw, ceil_div(rows, kBlock));  // a last, shorter chunk
      q.part_rows = vp, q.out_cols = (int)whole, q.scale = &head->scale_up;
      if (own) q.out = a.dw, q.ldo = a.lddw, q.out_end = (int)H;
      q.even = reinterpret_cast<uintptr_t>(a.dw) % 4 == 0 && a.lddw % 2 == 0;
      q.db = p.db ? reinterpret_cast<float*>(ws + p.db_sums) : nullptr;
      if (p.db_now) q.db_out = a.db, q.db32 = a.db_dtype == PSGD_F32;
      q.add = t0 > 0 || (p.direct && a.accumulate), q.db_add = t0 > 0;
      q.lost = &head->lost;
      if ((rc = p.half ? dense<T, kDw16>(call, ma, mb, mc, q) : dense<T, kDw>(call, ma, mb, mc, q))) return rc;
    }
    // dx reads what dw reads: it starts on the SMs that dw's last wave of tiles leaves idle
    if (p.dx) {
      CUtensorMap ma, mb, mc;
      float* part = reinterpret_cast<float*>(ws + p.part);
      const int64_t sc[2] = {H, p.px * padded};
      if ((rc = encode(&ma, dtype, e, 2, se, &p.lde, 128)) || (rc = encode(&mb, dtype, w.p, 2, sw, &lw, 64)) ||
          (rc = encode(&mc, PSGD_F32, part, 2, sc, &p.ldp, 32)))
        return rc;
      DenseArgs q = {};
      q.mdim = (int)rows, q.ndim = (int)H, q.depth = (int)V, q.width = p.nx, q.parts = p.px, q.part_rows = padded;
      q.out_cols = (int)H, q.beside = p.dw || p.db, q.lost = &head->lost;
      if ((rc = dense<T, kDx>(call, ma, mb, mc, q))) return rc;
      JoinArgs j = {};
      j.part = part, j.step = padded * p.ldp, j.parts = p.px, j.rows = rows, j.ldp = p.ldp, j.cols = (int)H;
      j.out = static_cast<T*>(a.dx) + t0 * a.lddx, j.ldo = a.lddx;
      j.aligned = reinterpret_cast<uintptr_t>(a.dx) % 8 == 0 && a.lddx % 4 == 0;
      j.factor = factor, j.head = head;
      if (last) j.loss = a.loss, j.losses = losses, j.all_rows = a.rows, j.mean = a.mean;
      const int64_t n = ceil_div(rows * (p.ldp / 4), 256);
      if ((rc = launch_behind(join_kernel<T>, dim3((unsigned)std::min<int64_t>(n, call.sms * 8)), 256, 0, stream, j)))
        return rc;
    }
  }
  if (!a.rows && !a.accumulate) {
    const size_t ws = a.dw_dtype == PSGD_F32 ? 4 : 2, bs = a.db_dtype == PSGD_F32 ? 4 : 2;
    if (p.dw) CUDA_TRY(cudaMemset2DAsync(a.dw, a.lddw * ws, 0, H * ws, V, stream));
    if (p.db) CUDA_TRY(cudaMemsetAsync(a.db, 0, V * bs, stream));
  }
  if (a.rows && p.dw && !p.direct && !p.half) {
    JoinArgs j = {};
    j.part = reinterpret_cast<const float*>(ws + p.sums), j.step = vp * p.ldw, j.parts = p.pw, j.rows = V, j.ldp = p.ldw;
    j.cols = (int)H, j.out = a.dw, j.ldo = a.lddw, j.add = a.accumulate, j.head = head;
    const int vec = a.dw_dtype == PSGD_F32 ? 16 : 8;
    j.aligned = reinterpret_cast<uintptr_t>(a.dw) % vec == 0 && a.lddw % 4 == 0;
    const int64_t n = ceil_div(V * (p.ldw / 4), 256);
    const dim3 grid((unsigned)std::min<int64_t>(n, call.sms * 8));
    rc = a.dw_dtype == PSGD_F32 ? launch_behind(join_kernel<float>, grid, 256, 0, stream, j)
                                : launch_behind(join_kernel<T>, grid, 256, 0, stream, j);
    if (rc) return rc;
  }
  const bool db = p.db && a.rows && !p.db_now, loss = a.loss && !a.rows;
  if (!loss && !db) return PSGD_OK;
  EndArgs e = {};
  e.losses = losses, e.rows = a.rows, e.loss = loss ? a.loss : nullptr, e.mean = a.mean;
  e.sums = reinterpret_cast<const float*>(ws + p.db_sums), e.step = vp, e.parts = p.pw, e.vocab = (int)V;
  e.db = db ? a.db : nullptr, e.add = a.accumulate, e.head = head;
  const dim3 grid((unsigned)(db ? std::min<int64_t>(ceil_div(V, 1024), call.sms) : 1));
  return db && a.db_dtype == PSGD_F32 ? launch_behind(end_kernel<float>, grid, 1024, 0, stream, e)
                                        : launch_behind(end_kernel<T>, grid, 1024, 0, stream, e);
}

int check(const Args* a) {
  if (!a) return fail(PSGD_ERR_INVALID, "the arguments must not be NULL");
  if (a->rows < 0 || a->rows > PSGD_MAX_EXPERT_ROWS)
    return fail(PSGD_ERR_INVALID, "rows must be in [0, %lld] (got %lld)", (long long)PSGD_MAX_EXPERT_ROWS, (long long)a->rows);
  if (a->vocab < 1 || a->vocab > PSGD_MAX_EXPERT_SIDE || a->width < 1 || a->width > PSGD_MAX_EXPERT_SIDE)
    return fail(PSGD_ERR_INVALID, "vocab and width must be in [1, %lld] (got %lld, %lld)", (long long)PSGD_MAX_EXPERT_SIDE,
                (long long)a->vocab, (long long)a->width);
  if (a->dtype != PSGD_BF16 && a->dtype != PSGD_F16)
    return fail(PSGD_ERR_INVALID, "the loss takes bfloat16 or float16 (got data type %d)", a->dtype);
  if (a->target_bytes != 4 && a->target_bytes != 8)
    return fail(PSGD_ERR_INVALID, "target has values of 4 or 8 bytes (got %d)", a->target_bytes);
  const auto own = [&](int32_t t) { return t == PSGD_F32 || t == a->dtype; };
  if ((a->bias && !own(a->bias_dtype)) || (a->dw && !own(a->dw_dtype)) || (a->db && !own(a->db_dtype)))
    return fail(PSGD_ERR_INVALID, "bias, dw and db are float32 or have the operands' type");
  return PSGD_OK;
}

// An address that is not NULL where it is needed, and aligned to its values.
int check_at(const char* name, const void* p, bool needed, int size) {
  if ((needed && !p) || reinterpret_cast<uintptr_t>(p) % size)
    return fail(PSGD_ERR_INVALID, "%s is NULL or not %d-byte aligned", name, size);
  return PSGD_OK;
}

int check_ld(const char* name, int64_t ld, int64_t least) {
  if (ld < least || ld > ((int64_t)1 << 40))
    return fail(PSGD_ERR_INVALID, "%s: row stride %lld is out of range", name, (long long)ld);
  return PSGD_OK;
}

}  // namespace
}  // namespace psgd

using namespace psgd;

extern "C" int psgd_cross_entropy_workspace(const psgd_cross_entropy_args* a, size_t* bytes) {
  const int rc = check(a);
  if (rc) return rc;
  if (!bytes) return fail(PSGD_ERR_INVALID, "bytes must not be NULL");
  *bytes = plan_of(*a).bytes;
  return PSGD_OK;
}

extern "C" int psgd_cross_entropy(const psgd_cross_entropy_args* args, void* workspace, size_t workspace_bytes,
                                  void* cuda_stream) {
  int rc = check(args);
  if (rc) return rc;
  const Args& a = *args;
  const bool any = a.rows > 0;
  const auto size = [](int32_t t) { return t == PSGD_F32 ? 4 : 2; };
  if ((rc = check_at("x", a.x, any, 2)) || (rc = check_at("w", a.w, any, 2)) ||
      (rc = check_at("target", a.target, any, a.target_bytes)) || (rc = check_at("bias", a.bias, false, size(a.bias_dtype))) ||
      (rc = check_at("row_scale", a.row_scale, false, 4)) || (rc = check_at("scale_dev", a.scale_dev, false, 4)) ||
      (rc = check_at("losses", a.losses, false, 4)) || (rc = check_at("loss", a.loss, false, 4)) ||
      (rc = check_at("dx", a.dx, false, 2)) || (rc = check_at("dw", a.dw, false, size(a.dw_dtype))) ||
      (rc = check_at("db", a.db, false, size(a.db_dtype))) || (rc = check_ld("x", a.ldx, 0)) ||
      (rc = check_ld("w", a.ldw, 0)) || (a.dx && (rc = check_ld("dx", a.lddx, a.width))) ||
      (a.dw && (rc = check_ld("dw", a.lddw, a.width))))
    return rc;
  const bool nothing = !a.losses && !a.loss && !a.dx && !a.dw && !a.db;
  if (any && nothing) return fail(PSGD_ERR_INVALID, "the call has no result");
  if (std::isnan(a.scale)) return fail(PSGD_ERR_INVALID, "scale must not be NaN");
  const Plan p = plan_of(a);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < p.bytes)
    return fail(PSGD_ERR_INVALID, "the loss needs a workspace of %zu bytes, 256-byte aligned (got %zu)", p.bytes,
                workspace ? workspace_bytes : (size_t)0);
  if (nothing) return PSGD_OK;  // results of no rows
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool wide = a.bias && a.bias_dtype == PSGD_F32;
  if (a.dtype == PSGD_BF16)
    return wide ? loss_of<__nv_bfloat16, float>(a, p, ws, s) : loss_of<__nv_bfloat16, __nv_bfloat16>(a, p, ws, s);
  return wide ? loss_of<__half, float>(a, p, ws, s) : loss_of<__half, __half>(a, p, ws, s);
}
