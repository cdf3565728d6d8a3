// Matrix products grouped by expert, with ragged group sizes.
//
// T rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1]-1
// and the matrix W[e] (N x K).
//   forward      y[t]  = W[e(t)] x[t]
//   grad_input   dx[t] = W[e(t)]^T dy[t]
//   grad_weight  dW[e] = sum over e's rows of dy[t] x[t]^T
// Products of bfloat16 or float16 values, float32 sums, one rounding at the end.
//
// One persistent kernel does the three: pairs of CTAs on the tensor cores, fed
// by TMA (below).  Around it: a copy of operands whose rows TMA cannot read,
// and the addition of contractions that were summed in parts.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>
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
  unsigned* abandoned = nullptr;  // where waits that run out are counted
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

// Warps that write results: the float32 sums of a weight gradient tile take 16
// (64 columns each; with 8 of 128 the writing held up tiles of few rows).
template <int OP>
constexpr int kWritersOf = OP == kGradWeight ? 16 : 8;
template <int OP>
constexpr int kPairThreads = (kWritersOf<OP> + 3) * 32;

// ------------------------------------------- pairs of CTAs, tcgen05 + TMA --
//
// The weights' output side is the MMA's M (256 rows a tile), the expert's rows
// (or, for the weight gradient, k) its N, which is chosen per tile: a ragged
// group costs only its own rows, rounded up to 32.
//   forward      D[n, t] = W[n, :] . x[t, :]      A K-major,  B K-major
//   grad_input   D[k, t] = W[:, k] . dy[t, :]     A MN-major, B K-major
//   grad_weight  D[n, k] = dy[:, n] . x[:, k]     A and B MN-major, over e's rows
// Roles of a CTA: the first 8 warps write results (each 32 rows of M by half of
// the columns; 16 warps by a quarter of them for grad_weight), the next loads,
// the next (leader) issues the MMAs, the last (grad_weight) clears the rows
// behind an expert's last one in the last block of its contraction.  Two
// accumulators of 256 columns let the results of a tile go out while the next
// is computed.
//
// The tensor cores truncate: of operands of one sign, an instruction loses
// 7.4e-8 of the sum in float16, whose products of 22 bits are cut one by one; in
// bfloat16 (16 bits) 7e-9 over the first 32, 2e-8 over 256 (4.8e-6 after 4096
// rows, where plain float32 has 6e-7) and as much as float16 in the end.  The
// weight gradient, float32 and as long as an expert has rows, therefore takes
// its sum out of TMEM every kRun blocks (512 rows) and adds the pieces in
// registers, rounded to nearest: 5.8e-7 on bfloat16 operands of one sign, 2.9e-6
// on float16 ones (4 blocks 1.4e-6, for 8 % of the training batch's time); on
// random ones 4.7e-7 and 6.4e-7.  More than kMostBlocks blocks (65536 rows, 128
// pieces) are summed as segments (longer ones of very large matrices, see
// cut_of).  What is added to a piece's error is then, of the sum of the terms'
// magnitudes, at most
//   128 pieces                   2^-24 x 129 / 2
//   S segments, in groups of 32  2^-24 x (33 + S / 32) / 2
// together 4.9e-6 for 2^20 rows of an expert, 5.1e-6 for 2^24.
//
// What bounds it: many rows an expert, the tensor cores; few rows, reading the
// weights (forward, input gradient) or writing them (weight gradient); a tile
// of 256 x 256 needs 64 bytes a clock of operands from L2 for each SM, so its
// stages are large and six deep (three were 2-10 % slower, four and five
// equal).  Measured with 8 experts of 8192 x 2048 and 32768 rows: 570-580 us
// forward (1896-1929 TFLOP/s, 1.00-1.01 of the measured 1900.6), 591 input
// gradient (0.98), 603-619 weight gradient (0.93-0.96) in short runs; under the
// power cap of long ones 671-700, 685-698 and 719-736 (1.57-1.64, 1.58-1.61 and
// 1.49-1.53 PFLOP/s of the sustained 1.73).  64 experts of 1024 x 2048 and 4096
// rows: 54 us forward (5.5 TB/s), 94 weight gradient (5.9 TB/s; 109 with eight
// writing warps; 120 with 16-bit results, whose variant for unaligned rows stores
// two bytes a lane).  One row each for 8 of 64 experts: 12 us on the device.
// What brought it there, on the first case: arrivals of relaxed order instead of release at cluster scope (each
// waited about 1 us for the thread's earlier stores) halved the time; single
// lanes elected inside warp-uniform loops instead of a divergent branch took
// 734 to 580 us; panels of 8 columns of tiles took the weight gradient from 755
// to 700, 16-byte stores of swapped register halves to 597.
constexpr int kMostStages = 6;
constexpr int kBlock = 64;                     // contraction values of a stage
constexpr int kSideBytes = 128 * kBlock * 2;   // one operand of one CTA and stage
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kChunkBytes = 64 * 128;          // 64 rows of an MN-major operand
constexpr int kBoxRows = 32;                   // rows of one load of the row operand
constexpr int kTileM = 256, kTileN = 256;
constexpr int kPanel = 8;                      // columns of tiles in a panel (in_panels)
constexpr int kRun = 8;                        // blocks between two readings of a weight gradient's sum
constexpr int kPatch = 32 * 32 * 2;             // a warp's staging of 32 x 32 results of 16 bits
constexpr int kRowPatch = 8 * 64 * 4;           // and of 8 x 64 float32 sums (STAGED)
constexpr uint32_t kNaN = 0x7FC00000u;         // what an abandoned tile's results are

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

// The device's counter, made on first use (also while a graph is captured).
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

// PSGD_ERR_TIMEOUT where products were abandoned that a stream's `waited` call
// (psgd_experts_sync) has not told this thread of, or a product's call nobody.
int report_abandoned(int device, const unsigned* count, cudaStream_t stream, bool waited) {
  std::atomic<unsigned>& told = g_abandoned[device].told;
  const unsigned now = *static_cast<const volatile unsigned*>(count), before = told.load(std::memory_order_relaxed);
  Seen& mine = seen_of(device, stream, before);
  if (now == (waited ? mine.count : before)) return PSGD_OK;
  mine.count = now;
  told.store(now, std::memory_order_relaxed);
  return fail(PSGD_ERR_TIMEOUT, waited ? "an expert product waited past its limit and was abandoned"
                                       : "an earlier expert product waited past its limit and was abandoned; nothing was "
                                         "enqueued for this one");
}

struct PairArgs {
  void* out;
  const int32_t* offsets;
  int64_t ldo, o_stride;
  int64_t rows;
  int experts;
  int mdim;   // result values along M
  int ndim;   // grad_weight: along N
  int depth;  // contraction (grad_weight: the expert's rows)
  bool aligned;   // 16-byte stores
  // a contraction summed in parts (see "Few tiles and a long contraction")
  int parts;        // forward, grad_input: of every tile; out is then float32
  int64_t part;     // values from one part's results to the next
  int seg, slots;   // grad_weight: blocks of a segment at most, and room for segments
  float* segments;  // their sums, slot_ld values a row
  int slot_ld;
  int width;        // forward, grad_input: most rows of a tile
  bool stall;       // tests: nothing is loaded, so that the waits run out
  uint32_t wait;    // limit of a wait, in units of 1024 ns
  unsigned* abandoned;  // counts waits that ran out
};

// Shared memory behind the stages.
struct PairShared {
  uint64_t full[kMostStages], empty[kMostStages], fix[kMostStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int stop;
  int groups;  // experts + 2: rows before the first expert and behind the last
  // then bound[groups + 1] (first row of each group), tile[groups + 1] (its
  // first row tile; grad_weight: its first segment) and, grad_weight,
  // slot[groups + 1] (where its segments' sums go)
};

// Stages of the ring, and bytes of staging for results behind them.
template <bool STAGED>
constexpr int kStagesOf = STAGED ? kMostStages - 1 : kMostStages;
template <int OP, bool STAGED>
constexpr int kPatches = kWritersOf<OP> * (OP != kGradWeight ? kPatch : STAGED ? kRowPatch : 0);

template <int OP, bool STAGED>
constexpr size_t pair_smem(int experts) {
  return 1024 + (size_t)kStagesOf<STAGED> * kStageBytes + kPatches<OP, STAGED> + sizeof(PairShared) +
         (size_t)(experts + 3) * (OP == kGradWeight ? 12 : 8);
}
static_assert(pair_smem<kForward, false>(kMaxExperts) <= 232448 && pair_smem<kGradWeight, false>(kMaxExperts) <= 232448 &&
                  pair_smem<kGradWeight, true>(kMaxExperts) <= 232448,
              "too large");

__host__ __device__ constexpr int up32(int v) { return (v + 31) & ~31; }

// One tile of the result.
struct Tile2 {
  int expert;     // -1: rows of no expert
  int row0;       // first row (grad_weight: of the expert)
  int m0;         // first value along M
  int n0, count;  // first value along N (rows are counted from row0) and how many
  int width;      // the MMA's N
  int d0;         // first contraction index
  int blocks;     // stages of the contraction; 0: the result is zero
  int last;       // contraction values in the last block
  int part;       // forward, grad_input: which part; grad_weight: slot of the segment's sum, -1: none
};

// The last of `groups` whose first tile is <= t (groups without tiles have the next one's).
__device__ __forceinline__ int group_of(const int* tile, int groups, int t) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

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
  const int* tile = bound + sh->groups + 1;
  const int mt = (p.mdim + kTileM - 1) / kTileM;
  Tile2 t;
  int depth, m, n, parts, part;
  if (OP == kGradWeight) {
    const int* slot = tile + sh->groups + 1;
    const int nt = (p.ndim + kTileN - 1) / kTileN;
    const int w = up32((p.ndim + nt - 1) / nt);
    const int q = idx / (mt * nt);
    in_panels(idx - q * (mt * nt), mt, nt, m, n);
    const int g = group_of(tile, sh->groups, q);
    t.expert = g - 1;
    t.n0 = n * w;
    t.count = min(w, p.ndim - t.n0);
    t.row0 = bound[g];
    depth = bound[g + 1] - t.row0;
    parts = tile[g + 1] - tile[g], part = q - tile[g];
    t.part = parts > 1 ? slot[g] + part : -1;
  } else {
    parts = p.parts, part = 0;
    if (parts > 1) {
      const int q = idx / parts;
      part = idx - q * parts, idx = q;
    }
    int tt;
    in_panels(idx, mt, tile[sh->groups], m, tt);
    const int g = group_of(tile, sh->groups, tt);
    const int c = bound[g + 1] - bound[g], nt = (c + p.width - 1) / p.width;
    const int w = up32((c + nt - 1) / nt);
    t.expert = g >= 1 && g <= p.experts ? g - 1 : -1;
    t.n0 = (tt - tile[g]) * w;
    t.count = min(w, c - t.n0);
    t.row0 = bound[g];
    depth = t.expert < 0 ? 0 : p.depth;
    t.part = part;
  }
  t.m0 = m * kTileM;
  t.width = up32(t.count);
  const int blocks = (depth + kBlock - 1) / kBlock;
  int b0 = 0, b1 = blocks;
  if (parts > 1) b0 = (int)((int64_t)blocks * part / parts), b1 = (int)((int64_t)blocks * (part + 1) / parts);
  t.d0 = b0 * kBlock;
  t.blocks = b1 - b0;
  t.last = b1 == blocks ? depth - (blocks - 1) * kBlock : kBlock;
  return t;
}

// Two float32 results, as bits, in 16 bits each (the first in the low half).
template <typename O>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
  alignas(4) const O v[2] = {from_f<O>(__uint_as_float(a)), from_f<O>(__uint_as_float(b))};
  return *reinterpret_cast<const uint32_t*>(v);
}

// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_sum(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(~0u, v, o);
    v += lane >= o ? u : 0;
  }
  return v;
}

// The groups of the offsets, 32 at a time and one a lane: f(i, begin, end)
// for group i = 0 .. experts (0: the rows before the first expert), with
// offsets outside [0, rows], or falling, taken as the nearest that are not.
// Returns the last expert's end.  One converged warp.
template <typename F>
__device__ __forceinline__ int each_group(const int32_t* offsets, int experts, int rows, F f) {
  const int lane = threadIdx.x & 31;
  int top = 0;
  int next = lane <= experts ? offsets[lane] : 0;
  for (int i0 = 0; i0 <= experts; i0 += 32) {
    const int i = i0 + lane;
    int end = i <= experts ? min(max(next, 0), rows) : 0;
    if (i + 32 <= experts) next = offsets[i + 32];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(~0u, end, o));  // lanes below o keep their own
    end = max(end, top);
    int begin = __shfl_up_sync(~0u, end, 1);
    if (lane == 0) begin = top;
    f(i, begin, end);
    top = __shfl_sync(~0u, end, 31);
  }
  return top;
}

// How the weight gradient's contractions are cut: running sums of segments
// and of slots over the groups.  An expert of more than `seg` blocks is cut
// into segments whose sums go to slots of their own.
struct Segments {
  int seg, slots;
  int done = 0, used = 0;  // segments and slots of the groups so far
  __device__ __forceinline__ Segments(int seg_, int slots_) : seg(seg_), slots(slots_) {}
  // one group a lane: its segments, the first of them, its first slot
  __device__ __forceinline__ void next(bool expert, int begin, int end, int& own, int& first, int& slot) {
    const int blocks = (end - begin + kBlock - 1) / kBlock;
    own = expert ? max(1, (blocks + seg - 1) / seg) : 0;
    int want = own > 1 ? own : 0;
    const int s = lane_sum(want);
    slot = used + s - want;
    used += __shfl_sync(~0u, s, 31);
    if (want && slot + want > slots) own = 1;  // no room: the host's bound leaves none out
    const int d = lane_sum(own);
    first = done + d - own;
    done += __shfl_sync(~0u, d, 31);
  }
};

// bound[], tile[] and slot[] from the offsets: one warp.
template <int OP>
__device__ __forceinline__ void scan_groups(const PairArgs& p, PairShared* sh) {
  const int E = p.experts, rows = (int)p.rows, lane = threadIdx.x & 31;
  int* bound = reinterpret_cast<int*>(sh + 1);
  int* tile = bound + E + 3;
  int* slot = tile + E + 3;
  Segments cut(p.seg, p.slots);
  int sum = 0;
  const int top = each_group(p.offsets, E, rows, [&](int i, int begin, int end) {
    int first, own, at;
    if (OP == kGradWeight) {
      cut.next(i >= 1 && i <= E, begin, end, own, first, at);
      sum = cut.done;
      if (i <= E) slot[i] = at;
    } else {
      own = (end - begin + p.width - 1) / p.width;
      const int s = lane_sum(own);
      first = sum + s - own;
      sum += __shfl_sync(~0u, s, 31);
    }
    if (i <= E) bound[1 + i] = end, tile[i] = first;
  });
  if (lane == 0) {
    bound[0] = 0, bound[E + 2] = rows;
    tile[E + 1] = sum, tile[E + 2] = sum + (OP == kGradWeight ? 0 : (rows - top + p.width - 1) / p.width);
    sh->groups = E + 2;
  }
}

// A warp's 32 x 64 sums of a weight gradient tile (pieces as in
// tmem_ld_16x32) to rows m0 .. of `out`, `left` columns of them; `rows` in all.
// STAGED: through shared memory, for 16-bit results and rows that do not start
// on 16-byte boundaries (kept apart: its registers cost the other form 15 % of
// a tile of few rows).  1539 rows, 20 of 1121 x 2151: 151 us value by value, 70
// so; 60 rows, 6 of 2137 x 7989 (410 MB) 113, 3.6 TB/s: a value a lane and store.
template <bool STAGED, typename O>
__device__ __forceinline__ void store_sums(O* out, int64_t ld, const float (&sum)[4][16], int m0, int rows, int left,
                                           float* patch) {
  const int lane = threadIdx.x & 31;
  if constexpr (STAGED) {
    if (left <= 0) return;
    // rows that start anywhere: eight at a time through shared memory, a value
    // each lane (row r there with its columns c at c ^ 8 (r % 4), free of bank
    // conflicts both ways)
    const int row = lane >> 2, mix = (row & 3) * 8;
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // rows 8 h .. + 7 of 32
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float2*>(patch + row * 64 + ((c * 32 + i * 8) ^ mix) + (lane & 3) * 2) =
              make_float2(sum[2 * c + (h >> 1)][4 * i + 2 * (h & 1)], sum[2 * c + (h >> 1)][4 * i + 2 * (h & 1) + 1]);
      __syncwarp();
      O* o = out + (int64_t)(m0 + 8 * h) * ld + lane;
      const int in = rows - m0 - 8 * h;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* from = patch + j * 64 + (lane ^ 8 * (j & 3));
        if (j < in && lane < left) o[j * ld] = from_f<O>(from[0]);
        if (j < in && lane + 32 < left) o[j * ld + 32] = from_f<O>(from[32]);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c0 = (q >> 1) * 32, mq = m0 + (q & 1) * 16;
      if (c0 >= left) continue;
      if (left - c0 >= 32) {
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
            if (m < rows)
              *reinterpret_cast<float4*>(o + (int64_t)m * ld + i * 8) =
                  odd ? make_float4(x, y, b0, b1) : make_float4(a0, a1, x, y);
          }
      } else {  // a row's last columns
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int m = mq + lane / 4 + r * 8;
          if (m >= rows) continue;
          O* row = out + (int64_t)m * ld;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + i * 8 + (lane & 3) * 2;
            if (c < left) row[c] = from_f<O>(sum[q][4 * i + 2 * r]);
            if (c + 1 < left) row[c + 1] = from_f<O>(sum[q][4 * i + 2 * r + 1]);
          }
        }
      }
    }
  }
}

// The same for an abandoned tile; out of line, to cost the others no registers.
template <typename O>
__device__ __noinline__ void store_nan(O* out, int64_t ld, int m0, int rows, int left) {
  for (int m = m0; m < min(m0 + 32, rows); ++m)
    for (int c = threadIdx.x & 31; c < min(left, 64); c += 32) out[(int64_t)m * ld + c] = from_f<O>(__uint_as_float(kNaN));
}

template <typename T, typename O, int OP, bool STAGED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads<OP>, 1)
    pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const PairArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kStages = kStagesOf<STAGED>;
  PairShared* sh = reinterpret_cast<PairShared*>(smem + kStages * kStageBytes + kPatches<OP, STAGED>);
  int* bound = reinterpret_cast<int*>(sh + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kAmn = OP != kForward, kBmn = OP == kGradWeight;
  constexpr int kWriters = kWritersOf<OP>;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init_count(&sh->full[s], 2);
      mbar_init_count(&sh->empty[s], 1);
      mbar_init_count(&sh->fix[s], 1);
    }
    for (int a = 0; a < 2; ++a) mbar_init_count(&sh->acc_full[a], 1), mbar_init_count(&sh->acc_empty[a], 2 * kWriters);
    sh->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWriters + 1) pair_tmem_alloc(&sh->tmem, 512);
  if (warp == kWriters && lane == 0) tma_prefetch_map(&map_a), tma_prefetch_map(&map_b);
  grid_wait();  // from here on the grids in front are done
  if (warp == 0) scan_groups<OP>(p, sh);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  const uint32_t tmem = sh->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = (bound + sh->groups + 1)[sh->groups] * ((p.mdim + kTileM - 1) / kTileM) *
                    (OP == kGradWeight ? (p.ndim + kTileN - 1) / kTileN : p.parts);
  const PairWait wait{&sh->stop, p.abandoned, p.wait};

  if (warp == kWriters) {
    // ---- loads
    const uint32_t base = smem_u32(smem);
    const uint32_t full0 = map_rank(smem_u32(&sh->full[0]), 0), fix0 = smem_u32(&sh->fix[0]);
    uint32_t s = 0, phase = 1;
    bool ok = true;
    for (int idx = pair; ok && !p.stall && idx < tiles; idx += pairs) {
      const Tile2 t = tile_at<OP>(p, sh, idx);
      const int half = t.width / 2;
      const int boxes = OP == kGradWeight ? (half + 63) / 64 : (half + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = kSideBytes + boxes * (OP == kGradWeight ? kChunkBytes : kBoxRows * 128);
      const int ma = t.m0 + (int)rank * 128, nb = t.n0 + (int)rank * half;
      for (int b = 0; b < t.blocks; ++b) {
        if (!(ok = __all_sync(~0u, pair_wait(&sh->empty[s], phase, wait)))) break;
        const bool ragged = OP == kGradWeight && b == t.blocks - 1 && (t.last & 15);
        const uint32_t bar = (ragged ? fix0 : full0) + s * 8;
        const uint32_t sa = base + s * kStageBytes, sb = sa + kSideBytes;
        const int d = t.d0 + b * kBlock;
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
          if (!(ok = __all_sync(~0u, pair_wait(&sh->acc_empty[a], (n >> 1 & 1) ^ 1, wait)))) break;
          tc_fence_after();
          const int end = min(r0 + run, t.blocks);
          for (int b = r0; b < end; ++b) {
            if (!(ok = __all_sync(~0u, pair_wait(&sh->full[s], phase, wait)))) break;
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
      // The next expert that ends inside 16 rows may be many tiles away, so this
      // is the one wait that a sound product can make long (all of a kernel of
      // seconds): it has 256 times the limit, and ends when another role's runs
      // out (the loads wait for a free stage, the results for every tile).
      const PairWait far{wait.stop, wait.abandoned, min(wait.limit, 1u << 23) * 256};
      uint32_t it = 0, phases = 0;
      bool ok = true;
      for (int idx = pair; ok && idx < tiles; idx += pairs) {
        const Tile2 t = tile_at<OP>(p, sh, idx);
        it += t.blocks;
        if (!t.blocks || !(t.last & 15)) continue;
        const int s = (it - 1) % kStages;
        if (!(ok = __all_sync(~0u, pair_wait(&sh->fix[s], phases >> s & 1, far)))) break;
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
    bool lost = false;  // a wait ran out: what is left to write is NaN (grad_weight asks sh->stop: no register is left)
    for (int idx = pair; idx < tiles; idx += pairs) {
      const Tile2 t = tile_at<OP>(p, sh, idx);
      const int m0 = t.m0 + (int)rank * 128 + quarter * 32;
      if (OP == kGradWeight) {
        // columns c0 .. + 63, in pieces of 16 rows x 32 columns (tmem_ld_16x32);
        // the first run's values start the sums
        const int c0 = half * 64, left = t.count - c0;
        float* patch = reinterpret_cast<float*>(smem + kStages * kStageBytes + warp * kRowPatch);
        float sum[4][16];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[q][j] = 0.f;
        for (int r0 = 0; r0 < t.blocks; r0 += kRun, ++n) {
          const uint32_t a = n & 1, from = tmem + a * kTileN + c0 + lanes;
          if (!__all_sync(~0u, pair_wait(&sh->acc_full[a], n >> 1 & 1, wait))) break;
          tc_fence_after();
          if (left > 0) {
            if (r0 == 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (q < 2 || left > 32) tmem_ld_16x32(from + (q >> 1) * 32 + ((uint32_t)((q & 1) * 16) << 16), sum[q]);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 4; ++q) hold(sum[q]);
            } else {
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                if (q && left <= 32) continue;
                uint32_t f[16], g[16];
                tmem_ld_16x32(from + (q >> 1) * 32, f);
                tmem_ld_16x32(from + (q >> 1) * 32 + (16u << 16), g);
                tmem_wait_ld(f, g);
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[q][j] += __uint_as_float(f[j]), sum[q + 1][j] += __uint_as_float(g[j]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_rank(smem_u32(&sh->acc_empty[a]), 0));
        }
        if (__any_sync(~0u, *wait.stop) && t.blocks) {  // some wait ran out, this warp's or another's
          if (t.part >= 0)
            store_nan(p.segments + (int64_t)t.part * p.mdim * p.slot_ld + t.n0 + c0, p.slot_ld, m0, p.mdim, left);
          else
            store_nan(static_cast<O*>(p.out) + t.expert * p.o_stride + t.n0 + c0, p.ldo, m0, p.mdim, left);
          continue;
        }
        if (t.part >= 0)
          store_sums<STAGED>(p.segments + (int64_t)t.part * p.mdim * p.slot_ld + t.n0 + c0, p.slot_ld, sum, m0, p.mdim, left,
                             patch);
        else
          store_sums<STAGED>(static_cast<O*>(p.out) + t.expert * p.o_stride + t.n0 + c0, p.ldo, sum, m0, p.mdim, left,
                             patch);
      } else {
        const uint32_t a = n & 1;
        if (t.blocks && !lost) {
          lost = !__all_sync(~0u, pair_wait(&sh->acc_full[a], n >> 1 & 1, wait));
          tc_fence_after();
        }
        const bool sums = t.blocks && !lost;  // in TMEM
        const uint32_t fill = t.blocks ? kNaN : 0;
        if constexpr (sizeof(O) == 4) {  // a part's sums, 128 bytes of a column at a time
          for (int c = half * 32; c < t.count; c += 64) {
            float f[32];
            if (sums) {
              tmem_ld32(tmem + a * kTileN + c + lanes, f);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(fill);
            }
            float* o = static_cast<float*>(p.out) + t.part * p.part + (int64_t)(t.row0 + t.n0 + c) * p.ldo + m0 + lane;
            if (m0 + lane < p.mdim) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c + j < t.count) o[j * p.ldo] = f[j];
            }
            __syncwarp();
          }
        } else {
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
            if (sums) {
              tmem_ld_16x32(tmem + a * kTileN + c + lanes, f);
              tmem_ld_16x32(tmem + a * kTileN + c + lanes + (16u << 16), g);
              tmem_wait_ld(f, g);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) f[j] = g[j] = fill;
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
        }
        if (sums) {
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

// Few tiles and a long contraction leave most SMs idle.  Then the contraction
// is summed in parts, float32 sums in the workspace that a second kernel adds
// in order.  How a product is cut depends on its sizes alone.
constexpr int kPairs = 76;        // pairs of CTAs on the device's 152 SMs
constexpr int kPartBlocks = 16;   // fewest blocks of a part or segment
constexpr int kLongBlocks = 96;   // a long contraction
// blocks that are summed in one piece at most (where there is room)
constexpr int kMostBlocks = 1024;                                                     // grad_weight
constexpr int most_blocks(int dtype) { return dtype == PSGD_F16 ? 512 : 4096; }       // forward, grad_input
struct Cut {
  int parts = 1;          // forward, grad_input: of every contraction
  int seg = 1 << 30;      // grad_weight: blocks of a segment at most
  int slots = 0;          // room for segments
  int64_t ld = 0;         // float32 values of a row of the sums
  size_t bytes = 0;
};

// Forward and grad_input: where the tiles fill at most half of the pairs, as
// many parts as fill them, each of kPartBlocks blocks or more.  A call, host
// and all, of 8 or 300 rows and a contraction of 4096: 20 us in one piece, 22
// in parts; of 8192: 30 against 23, and 2000 rows by 1024: 41 against 32.
// However many the tiles, a part has most_blocks blocks at most: the sum stays in
// TMEM to a part's end, and what it loses there (7.4e-8 an instruction, see
// above) is then under a third of the rounding to 16 bits: 1.5e-4 of 4.9e-4 over
// 32768 values of float16, 1.2e-3 of 3.9e-3 over 262144 of bfloat16.
//
// grad_weight: an expert of more blocks than 1.5 shares of the device (so that
// equal experts that nearly fill it stay whole: cut in two, 4 of 1024 x 1024
// took 58 us for 44) is cut into segments, whatever the others have; where the
// experts' tiles fill the device by themselves, only from kLongBlocks in all on
// (the adding kernel costs 3 us, cut or not).  One expert of 512 x 512 with
// 30000 rows: 132 -> 28 us, with 4000 25 -> 16.  With T / 64
// blocks in all, an expert that is cut has over `seg` of them, so there are at
// most T / 64 / seg such, of at most (T / 64 + their number) / seg + their
// number segments: the bound on slots.  For the sake of its rounding (see
// above) a segment has kMostBlocks at most, or as much more as brings the
// segments' sums down to a quarter of the memory that the product has anyway:
// twice that for one expert of 16384 x 16384.
template <int OP>
Cut cut_of(int64_t rows, int experts, int64_t n, int64_t k, int dtype) {
  Cut c;
  const int64_t mdim = OP == kGradInput ? k : n, mt = ceil_div(mdim, kTileM);
  if (OP == kGradWeight) {
    const int64_t per = mt * ceil_div(k, kTileN), all = ceil_div(rows, kBlock);
    int64_t seg = std::max<int64_t>(kPartBlocks, ceil_div(per * all * 3, kPairs * 2));
    if (all <= kMostBlocks && (all <= seg || (all < kLongBlocks && experts * per >= kPairs))) return c;
    c.ld = (k + 3) / 4 * 4;
    const auto slots = [&](int64_t s) { return (all + all / s) / s + all / s + 1; };
    const int64_t room = (rows * (n + k) * 2 + experts * n * k * 4) / 4;
    int64_t exact = kMostBlocks;
    while (exact < all && slots(exact) * n * c.ld * 4 > room) exact *= 2;
    seg = std::min(seg, exact);
    if (all <= seg) return Cut();
    c.seg = (int)seg;
    c.slots = (int)slots(seg);
    c.bytes = (size_t)c.slots * n * c.ld * 4;
  } else {
    const int64_t blocks = ceil_div(OP == kForward ? k : n, kBlock);
    const int64_t tiles = mt * (rows / kTileN + std::min<int64_t>(experts, rows));
    int64_t parts = blocks < kLongBlocks ? 1 : std::min(kPairs / std::max<int64_t>(tiles, 1), blocks / kPartBlocks);
    parts = std::max(parts, ceil_div(blocks, most_blocks(dtype)));
    if (parts < 2) return c;
    c.parts = (int)parts;
    c.ld = (mdim + 3) / 4 * 4;
    c.bytes = (size_t)parts * rows * c.ld * 4;
  }
  c.bytes = (c.bytes + 255) / 256 * 256;
  return c;
}

// The sum of four values at each of `count` places, `step` apart.
__device__ __forceinline__ float4 sum_rows(const float* at, int64_t step, int count) {
  float4 s = *reinterpret_cast<const float4*>(at);
#pragma unroll 4
  for (int p = 1; p < count; ++p) {
    const float4 v = *reinterpret_cast<const float4*>(at + p * step);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  return s;
}

// y = the sum of a product's parts, four values a thread and step.
template <typename T>
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float* part, int64_t step, int parts, T* out, int64_t rows, int cols, int64_t ldp, int64_t ldo,
                     bool aligned) {
  grid_wait();
  const int vecs = (int)(ldp / 4);
  const int64_t n = rows * vecs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = n < ((int64_t)1 << 32) ? (uint32_t)i / (uint32_t)vecs : i / vecs;
    const int c = (int)(i - row * vecs) * 4;
    const float* at = part + row * ldp + c;
    const float4 s = sum_rows(at, step, parts);
    T* o = out + row * ldo + c;
    alignas(8) const T v[4] = {from_f<T>(s.x), from_f<T>(s.y), from_f<T>(s.z), from_f<T>(s.w)};
    if (aligned && c + 4 <= cols) {
      *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < cols) o[j] = v[j];
    }
  }
}

// dW of the experts whose contraction was cut: blockIdx.y counts them.
template <typename O>
__global__ void __launch_bounds__(256)
    sum_segments_kernel(const float* sums, const int32_t* offsets, int experts, int rows, int seg, int slots, O* out, int n,
                        int k, int64_t lds, int64_t ldo, int64_t o_stride, bool aligned) {
  __shared__ int s_expert, s_slot, s_own;
  grid_wait();
  if (threadIdx.x == 0) s_own = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    Segments cut(seg, slots);
    int before = 0;  // cut experts so far
    each_group(offsets, experts, rows, [&](int i, int begin, int end) {
      int own, first, slot;
      cut.next(i >= 1 && i <= experts, begin, end, own, first, slot);
      const unsigned many = __ballot_sync(~0u, own > 1);
      if (own > 1 && before + __popc(many & ((1u << (threadIdx.x & 31)) - 1u)) == (int)blockIdx.y)
        s_expert = i - 1, s_slot = slot, s_own = own;
      before += __popc(many);
    });
  }
  __syncthreads();
  const int own = s_own;
  if (!own) return;
  const int vecs = (int)(lds / 4);
  const int64_t step = (int64_t)n * lds, total = (int64_t)n * vecs;
  const float* base = sums + s_slot * step;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = total < ((int64_t)1 << 32) ? (uint32_t)i / (uint32_t)vecs : i / vecs;
    const int c = (int)(i - row * vecs) * 4;
    const float* at = base + row * lds + c;
    float4 s = sum_rows(at, step, min(own, 32));
    for (int p = 32; p < own; p += 32) {  // by groups of 32: fewer roundings of large sums
      const float4 g = sum_rows(at + p * step, step, min(own - p, 32));
      s.x += g.x, s.y += g.y, s.z += g.z, s.w += g.w;
    }
    O* o = out + s_expert * o_stride + row * ldo + c;
    const float v[4] = {s.x, s.y, s.z, s.w};
    if (sizeof(O) == 4 && aligned && c + 4 <= k) {
      *reinterpret_cast<float4*>(o) = s;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < k) o[j] = from_f<O>(v[j]);
    }
  }
}

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

// Most rows of a tile: 256, or fewer where whole waves of 256 leave many pairs
// idle and the tiles are few enough to be foreseen from equal groups (ragged
// ones add or spare less than half a wave).  A tile costs a part of its own
// (the weights' side) and one that goes with its rows: 150 ns and 0.7 ns a row
// for a stage, fitted to widths of 64 to 256.  2 experts of 2048 x 2048, 3000
// rows: 25 us with 256, 21 with the width chosen here.
int rows_width(int64_t rows, int experts, int64_t mt, int parts, int pairs) {
  if (experts * mt * parts * 2 > pairs || rows > ((int64_t)1 << 24)) return kTileN;
  int width = kTileN;
  double best = 0;
  for (int w = kTileN; w >= 128; w -= 32) {
    const int64_t group = ceil_div(rows, experts), tiles = experts * ceil_div(group, w);
    const double cost = (double)ceil_div(tiles * mt * parts, pairs) * (150.0 + 0.7 * (double)rows / (double)tiles);
    if (w == kTileN || cost < best) best = w == kTileN ? 0.93 * cost : cost, width = w;
  }
  return width;
}

// Tiles of a product at most, whatever its offsets.
template <int OP>
int64_t most_tiles(const ProductArgs& p, const Cut& cut) {
  const int64_t mt = ceil_div(OP == kGradInput ? p.k : p.n, kTileM);
  return OP == kGradWeight ? (p.experts + cut.slots) * mt * ceil_div(p.k, kTileN)
                           : cut.parts * mt * (p.rows / 128 + std::min<int64_t>(p.experts + 2, p.rows));
}

template <typename T, typename O, int OP, bool STAGED = false>
int launch_pair(const ProductArgs& p, int dtype, const Cut& cut, float* sums, cudaStream_t stream) {
  static thread_local uint64_t ready = 0;
  int dev = 0, sms = 0, rc;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  auto kernel = pair_kernel<T, O, OP, STAGED>;
  if ((rc = allow_smem(kernel, pair_smem<OP, STAGED>(kMaxExperts), dev, &ready))) return rc;
  CUtensorMap ma, mb;
  const int64_t acols = OP == kForward ? p.k : p.n;
  const int64_t lda = tma_stride(p.lda, acols, p.rows);
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
  PairArgs a = {};
  a.out = p.c, a.offsets = p.offsets, a.ldo = p.ldc, a.o_stride = p.c_stride, a.rows = p.rows, a.experts = p.experts;
  a.mdim = OP == kGradInput ? p.k : p.n;
  a.ndim = p.k;
  a.depth = OP == kForward ? p.k : p.n;
  a.wait = (uint32_t)((uint64_t)g_wait_ms.load(std::memory_order_relaxed) * 1000000u >> 10);
  a.stall = t_stall;
  a.abandoned = p.abandoned;
  a.parts = cut.parts, a.seg = cut.seg, a.slots = cut.slots, a.segments = sums, a.slot_ld = (int)cut.ld;
  if (cut.parts > 1) a.out = sums, a.ldo = cut.ld, a.part = p.rows * cut.ld;
  const int vec = 16 / sizeof(O);
  a.aligned = reinterpret_cast<uintptr_t>(p.c) % (vec * sizeof(O)) == 0 && p.ldc % vec == 0 && p.c_stride % vec == 0;
  const int64_t mt = ceil_div(a.mdim, kTileM);
  a.width = rows_width(p.rows, p.experts, mt, cut.parts, sms / 2);
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(sms / 2, most_tiles<OP>(p, cut)));
  return launch_behind(kernel, dim3((unsigned)(2 * pairs)), kPairThreads<OP>, pair_smem<OP, STAGED>(p.experts), stream, ma, mb, a);
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
int make_readable(Operand* a, Operand* b, const int32_t* offsets, unsigned char* ws, cudaStream_t stream) {
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
  copy_kernel<<<dim3((unsigned)std::min<int64_t>(ceil_div(most, 256 * kCopies), most_ctas), (unsigned)experts), 256, 0,
                stream>>>(m[0], m[1], offsets);
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
  const size_t copies = copy_bytes(a) + copy_bytes(b);
  const size_t room = p.ws && reinterpret_cast<uintptr_t>(p.ws) % 256 == 0 ? p.ws_bytes : 0;
  Cut cut = cut_of<OP>(p.rows, p.experts, p.n, p.k, dtype);
  if (room < copies + cut.bytes) cut = Cut();
  // every refusal comes before the first launch
  if (room < copies)
    return fail(PSGD_ERR_INVALID, "operands whose rows do not start on 16-byte boundaries need a workspace of %zu bytes, "
                "256-byte aligned (got %zu)", copies, p.ws ? p.ws_bytes : (size_t)0);
  if (const int64_t most = most_tiles<OP>(p, cut); most > INT32_MAX / 2)
    return fail(PSGD_ERR_INVALID, "the product has too many tiles (%lld)", (long long)most);
  int dev = 0, rc;
  CUDA_TRY(cudaGetDevice(&dev));
  if ((rc = abandoned_of(dev, &p.abandoned)) || (rc = report_abandoned(dev, p.abandoned, s, false))) return rc;
  if ((rc = make_readable(&a, &b, p.offsets, p.ws, s))) return rc;
  p.a = a.p, p.lda = a.ld, p.b = b.p, p.ldb = b.ld, p.b_stride = b.stride;
  float* sums = reinterpret_cast<float*>(p.ws + copies);
  if constexpr (OP == kGradWeight) {
    const bool aligned = reinterpret_cast<uintptr_t>(p.c) % 16 == 0 && p.ldc % 4 == 0 && p.c_stride % 4 == 0;
    if constexpr (sizeof(O) == 4)
      rc = aligned ? launch_pair<T, O, OP>(p, dtype, cut, sums, s) : launch_pair<T, O, OP, true>(p, dtype, cut, sums, s);
    else
      rc = launch_pair<T, O, OP, true>(p, dtype, cut, sums, s);
    if (rc || !cut.slots) return rc;
    const int64_t steps = ceil_div((int64_t)p.n * (cut.ld / 4), 256), many = std::max(1, cut.slots / 2);
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(steps, 152 * 8 / many));
    return launch_behind(sum_segments_kernel<O>, dim3((unsigned)ctas, (unsigned)many), 256, 0, s, static_cast<const float*>(sums), p.offsets, p.experts, (int)p.rows, cut.seg, cut.slots,
                         static_cast<O*>(p.c), p.n, p.k, cut.ld, p.ldc, p.c_stride, aligned);
  } else {
    if (cut.parts == 1) return launch_pair<T, O, OP>(p, dtype, cut, sums, s);
    if ((rc = launch_pair<T, float, OP>(p, dtype, cut, sums, s))) return rc;
    const int cols = OP == kGradInput ? p.k : p.n;
    const bool aligned = reinterpret_cast<uintptr_t>(p.c) % 8 == 0 && p.ldc % 4 == 0;
    return launch_behind(sum_parts_kernel<O>,
                         dim3((unsigned)std::min<int64_t>(ceil_div(p.rows * (cut.ld / 4), 256), 152 * 8)), 256, 0, s,
                         static_cast<const float*>(sums), p.rows * cut.ld, cut.parts, static_cast<O*>(p.c), p.rows, cols,
                         cut.ld, p.ldc, aligned);
  }
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
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_stride(w_stride)) ||
      (rc = check_matrix("y", y, rows, 2, ldy, n, true)))
    return rc;
  const ProductArgs p{x, w, y, offsets, ldx, ldw, ldy, w_stride, 0, rows, experts, (int)n, (int)k,
                      static_cast<unsigned char*>(workspace), workspace_bytes};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == PSGD_BF16 ? product<__nv_bfloat16, __nv_bfloat16, kForward>(p, dtype, s)
                            : product<__half, __half, kForward>(p, dtype, s);
}

extern "C" int psgd_experts_grad_input(int64_t rows, int experts, int64_t n, int64_t k, int dtype, const void* dy,
                                       int64_t lddy, const void* w, int64_t ldw, int64_t w_stride,
                                       const int32_t* offsets, void* dx, int64_t lddx, void* workspace,
                                       size_t workspace_bytes, void* cuda_stream) {
  int rc = check(rows, experts, n, k, dtype);
  if (rc || (rc = check_offsets(offsets)) || (rc = check_matrix("dy", dy, rows, 2, lddy, n, false)) ||
      (rc = check_matrix("w", w, 1, 2, ldw, k, false)) || (rc = check_stride(w_stride)) ||
      (rc = check_matrix("dx", dx, rows, 2, lddx, k, true)))
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
  return out_dtype == PSGD_F32 ? product<__half, float, kGradWeight>(p, dtype, s)
                               : product<__half, __half, kGradWeight>(p, dtype, s);
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
  const int dtype = PSGD_F16;  // makes use of the most
  const Cut cut = op == kForward     ? cut_of<kForward>(rows, experts, n, k, dtype)
                  : op == kGradInput ? cut_of<kGradInput>(rows, experts, n, k, dtype)
                                     : cut_of<kGradWeight>(rows, experts, n, k, dtype);
  *bytes = rows ? copy_bytes(oa) + copy_bytes(ob) + cut.bytes : 0;
  return PSGD_OK;
}

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
