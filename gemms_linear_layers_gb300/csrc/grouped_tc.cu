// grouped_tc.cu -- the three products of a linear layer whose rows are
// grouped by expert, on tcgen05 CTA pairs.
//
// Rows [offsets[e], offsets[e+1]) of the activations belong to expert e:
//   forward          Y[t]  = X[t] W[e]^T
//   input gradient   dX[t] = dY[t] W[e]
//   weight gradient  dW[e] = sum over the rows t of e of dY[t]^T X[t]
// The offsets are read on the device, so no call waits for the host and a
// captured call follows new offsets.
//
// Which operand is the 256-row side of the MMA.  tcgen05.mma takes M = 256
// for a pair whatever the data, but N is any multiple of 32 up to 256.  A
// group's row count is the ragged size, so in the forward and input-gradient
// products the WEIGHT rows (or columns) are M and the group's rows are N:
// the kernel computes Y^T tiles of 256 features x up to 256 rows, a group of n
// rows costs ceil(n / 32) * 32 columns of MMA instead of ceil(n / 256) * 256,
// and each expert's weight is streamed once when its rows fit one tile.  A
// group of more rows is cut into tiles of nearly equal width.  Rows of a
// neighbouring group that a load box takes in end in accumulator columns that
// are never stored, so whatever they hold (NaN too) stays with them.
//
// In the weight gradient the ragged size is the reduction.  Whole 16-row slices
// of a group go through the ring (the MMAs of its last 64-row block stop at the
// last of them).  What is left, up to 15 rows, comes with rows of the next group
// that must not reach the sums: that slice is loaded into a small buffer of its
// own, a "mender" warp of each CTA overwrites the foreign rows with zeros in both
// operands (zeroing one only would leave 0 * NaN), and the MMA takes it last.
// The slice is requested before the group's blocks, so mending it costs no time
// once a group has a few blocks: mended in the ring, 8 uneven groups of 4,096
// rows (2,304 x 5,760) took 92 us; with all sizes multiples of 16, 78.
//
// Roles of a CTA (7 warps): 0 producer (TMA), 1 MMA issuer (rank 0 of the
// pair), 2-5 epilogue, 6 mender (weight gradient).  Every wait is bounded.  Two last
// as long as reductions do, the epilogue's for an accumulator and the mender's for the
// next slice: their bound grows with the blocks in between (10^9 rows of one expert in
// a unit take 3 to 4 s, the plain bound is 2).
//
// Bound by the MMA rate and L2 while groups have hundreds of rows, by HBM
// (weights) below; the weight gradient of small groups by its epilogue's stores.
// Measured: one group of 4,096 rows, 5,760 -> 2,304: 1,830 / 1,790 / 1,760 TFLOP/s
// forward / input gradient / weight gradient; 16,384 rows over 64 experts, 2,304 ->
// 5,760: 335 to 349 us at full clocks (1,240 to 1,290 TFLOP/s, 5.6 to 5.9 TB/s), 363 to
// 383 in rows of hundreds of calls and more, where the power limit lowers the clocks;
// 64 rows over 8 experts: 35 us, 6 TB/s; 8 uneven groups of 4,096 rows: 82 to 100 us
// input gradient (162 tiles for 76 pairs), 81 to 90 us weight gradient (ranges over GPUs
// and sessions); one row of one small expert: 4.2 us.
#include <cuda.h>
#include <stdio.h>

#include "grouped.h"
#include "pitch_copy.cuh"
#include "ptx.cuh"
#include "smem_attr.h"

namespace tg {
namespace {

constexpr int G_FWD = 0, G_DGRAD = 1, G_WGRAD = 2;

constexpr int GT_THREADS = 224;
constexpr int GT_BM = 256;        // rows of the pair's tile
constexpr int GT_BN = 256;        // largest tile width
constexpr int GT_BK = 64;
constexpr int GT_STAGES = 6;
constexpr int GT_A_BYTES = 128 * GT_BK * 2;  // one CTA's operand halves of a stage
constexpr int GT_B_BYTES = 128 * GT_BK * 2;
constexpr int GT_SLICES = 2;      // weight gradient: buffers of a group's last 16-row slice
constexpr int GT_SLICE_BYTES = 4 * 16 * 128;  // two 64-column chunks of each operand
constexpr int GT_MAXG = GROUPED_PER_LAUNCH + 2;   // experts of a launch, rows before and after them
constexpr int GT_BAR_BYTES = 384;
constexpr unsigned long long GT_BLOCK_NS = 8000;  // most that a block of a reduction may take (0.2 to 0.3 us measured)
constexpr int GT_SPLIT_SAVES = 20;  // blocks that splitting reductions has to save a pair

template <int OP>
struct GtCfg {
  static constexpr int SLICES = OP == G_WGRAD ? GT_SLICES * GT_SLICE_BYTES : 0;
  static constexpr int TURN = OP == G_WGRAD ? 4 * 32 * 33 * 4 : 0;  // 32 x 32 values of each epilogue warp
  static constexpr int TAB = (GT_MAXG + 1) * 4 * (OP == G_WGRAD ? 1 : 2);
  static constexpr int SMEM = 1024 + GT_STAGES * (GT_A_BYTES + GT_B_BYTES) + SLICES + TURN + GT_BAR_BYTES + TAB;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((2 * GT_STAGES + 3 * GT_SLICES + 5) * 8 + 16 <= GT_BAR_BYTES, "barrier area");
};

struct GtArgs {
  const int* offsets;  // [E + 1]
  void* out;
  long long T;
  int E;           // experts of this launch
  int M;           // forward: d_out; input gradient: d_in; weight gradient: d_out
  int N;           // weight gradient: d_in
  int K;           // forward: d_in; input gradient: d_out
  int m_tiles;     // of 256
  float by_m, by_tiles;  // 1 / m_tiles, 1 / (m_tiles n_tiles)
  int n_tiles;     // weight gradient: column tiles
  int n_width;     // weight gradient: width of a column tile (a multiple of 64)
  int ksplit;      // every tile's reduction in so many ranges, FP32 sums of each to out [ksplit][..]
  int first, last; // this launch holds the first / last experts: it zeroes the rows outside every group
  int out_kind;
  int wide;        // forward, input gradient: two 16-bit features in one store; weight gradient: 32-byte stores
  int pair_out;    // weight gradient without `wide`: 16-bit, an even width, 4-byte aligned
  uint32_t idesc;  // without N
  unsigned long long timeout_ns;
  unsigned int* status;
};

struct GtMaps {
  CUtensorMap A;     // forward: W (box 64 x 128 rows); input gradient: W (64 x 64); weight gradient: dY (64 x 64)
  CUtensorMap B[4];  // forward, input gradient: rows in boxes of 128, 64, 32, 16; weight gradient: [0] = X (64 x
                     // 64), and boxes of 16 rows for the slices: [1] = dY, [2] = X
};

// One unit of work: a tile of one group.
struct GtUnit {
  int m0;    // first feature row of the pair's tile
  int n0;    // first column: row of the activations, or (weight gradient) column of dW
  int n;     // columns that are stored; 0 or less: nothing to do
  int nmma;  // columns the MMA computes (a multiple of 32)
  int e;     // expert (index of this launch)
  int r0;    // weight gradient: first row of the reduction
  int s;     // range of the reduction
  int kb;    // 64-deep blocks of the reduction (weight gradient: of whole 16-row slices)
  int k0, k1;  // those of this range
  int tail;  // 16-deep slices of the last block, 1..4
  int rest;  // weight gradient: rows in the last slice (0: none, or all 16 in a block, or in another range)
  __device__ __forceinline__ bool zero() const { return k0 == k1 && rest == 0; }  // an empty sum
};

__device__ __forceinline__ int pairs_in_grid() { return static_cast<int>(gridDim.x >> 1); }

// Group tables in shared memory.  off[0 .. E]: the launch's offsets, made
// non-decreasing and confined to [0, T] (so that offsets that break the rules
// still address nothing outside the tensors).  Forward and input gradient:
// group 0 holds the rows before the first expert, 1..E the experts, E + 1 the
// rows after the last; start[g] = first row, cum[g] = units before group g.
template <int OP>
struct GtTab {
  int* off;  // weight gradient: off[0..E]; otherwise start[0..E+2]
  int* cum;  // forward, input gradient
  int units;
  // Forward, input gradient: the tiles of the last round, when they are at most
  // half the pairs, are cut into `cuts` narrower ones each, so that the round
  // ends sooner (8 uneven groups of 4,096 rows, 2,304 features: 162 tiles for 76 pairs).
  int whole, cuts;  // units of the rounds before it
};

// n / d for 0 <= n < 2^31, by = 1 / d rounded: the integer divisions' dozens of
// dependent instructions stood between a unit and its first copy (1,000 rows over 32
// experts 19.3 us with them, 17.3 without).  The estimate is off by at most 2^-22 of
// itself (four roundings), so while the quotient is at most 2^22 its floor is off by
// one at most.  It is an expert of 256, or a tile along the rows or columns of a result:
// more than 2^22 of these beside two or more feature tiles would be a tensor of more
// than 2^38 elements, which the entry points refuse; beside one, d = 1 and n < 2^24:
// exact.
__device__ __forceinline__ int quotient(int n, int d, float by) {
  int q = __float2int_rd(__int2float_rn(n) * by);
  const int r = n - q * d;
  if (r < 0) --q;
  if (r >= d) ++q;
  return q;
}
__device__ __forceinline__ int tiles_of(int rows) { return (rows + GT_BN - 1) / GT_BN; }

template <int OP>
__device__ void gt_build(const GtArgs& a, GtTab<OP>& t, int* s_plan) {
  // one warp: running maximum of the clamped offsets, then (forward, input
  // gradient) running sum of the groups' unit counts
  const int lane = threadIdx.x & 31;
  const int T = static_cast<int>(a.T);
  const int shift = OP == G_WGRAD ? 0 : 1;
  int run = 0;
  for (int b = 0; b <= a.E; b += 32) {
    const int i = b + lane;
    int v = i <= a.E ? min(max(a.offsets[i], 0), T) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v = max(v, w);
    }
    v = max(v, run);
    if (i <= a.E) t.off[i + shift] = v;
    run = __shfl_sync(~0u, v, 31);
  }
  __syncwarp();
  if (OP == G_WGRAD) {
    if (lane == 0) s_plan[0] = a.E * a.m_tiles * a.n_tiles * a.ksplit;
    return;
  }
  if (lane == 0) {
    // rows outside every group: only the launches with the first and last experts own them
    t.off[0] = a.first ? 0 : t.off[1];
    t.off[a.E + 2] = a.last ? T : t.off[a.E + 1];
  }
  __syncwarp();
  const int G = a.E + 2;
  int sum = 0;
  for (int b = 0; b < G; b += 32) {
    const int g = b + lane;
    const int u = g < G ? tiles_of(t.off[g + 1] - t.off[g]) * a.m_tiles : 0;
    int v = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += w;
    }
    if (g < G) t.cum[g] = sum + v - u;
    sum += __shfl_sync(~0u, v, 31);
  }
  if (lane == 0) {
    t.cum[G] = sum;
    // the last round
    const int pairs = pairs_in_grid();
    int whole = 0, tail = sum, cuts = 1;
    if (sum >= pairs) {
      whole = sum / pairs * pairs;
      tail = sum - whole;
      if (tail > 0 && a.ksplit == 1) cuts = min(pairs / tail, GT_BN / 32);
    }
    s_plan[0] = a.ksplit > 1 ? sum * a.ksplit : whole + tail * cuts;
    s_plan[1] = whole;
    s_plan[2] = cuts;
  }
}

template <int OP>
__device__ __forceinline__ GtUnit gt_unit(const GtArgs& a, const GtTab<OP>& t, int u) {
  GtUnit c;
  c.s = 0;
  if (a.ksplit > 1) {
    const int t = u / a.ksplit;
    c.s = u - t * a.ksplit;
    u = t;
  }
  if (OP == G_WGRAD) {
    const int per = a.m_tiles * a.n_tiles;
    c.e = quotient(u, per, a.by_tiles);
    const int r = u - c.e * per;
    const int nt = quotient(r, a.m_tiles, a.by_m);
    c.m0 = (r - nt * a.m_tiles) * GT_BM;
    c.n0 = nt * a.n_width;
    c.n = min(a.n_width, a.N - c.n0);
    c.nmma = (c.n + 63) / 64 * 64;
    c.r0 = t.off[c.e];
    const int rows = t.off[c.e + 1] - c.r0;
    const int slices = rows >> 4;
    c.rest = rows & 15;
    c.kb = (slices + 3) >> 2;
    c.tail = slices - (c.kb - 1) * 4;
  } else {
    int cut = 0;
    if (u >= t.whole) {
      const int v = u - t.whole, w = t.cuts == 1 ? v : v / t.cuts;
      cut = v - w * t.cuts;
      u = t.whole + w;
    }
    int lo = 0, hi = a.E + 1;  // the last group whose units start at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.cum[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    const int start = t.off[lo], rows = t.off[lo + 1] - start;
    const int r = u - t.cum[lo];
    const int nt = quotient(r, a.m_tiles, a.by_m);
    const int tiles = tiles_of(rows);
    const int width = ((tiles <= 1 ? rows : (rows + tiles - 1) / tiles) + 31) / 32 * 32;
    c.m0 = (r - nt * a.m_tiles) * GT_BM;
    c.n0 = start + nt * width;
    c.n = min(width, rows - nt * width);
    if (u >= t.whole && t.cuts > 1) {
      const int part = ((c.n + t.cuts - 1) / t.cuts + 31) / 32 * 32;
      c.n0 += cut * part;
      c.n = min(part, c.n - cut * part);  // nothing is left for the last cuts of a narrow tile
    }
    c.nmma = (c.n + 31) / 32 * 32;
    c.e = lo - 1;
    const bool expert = lo >= 1 && lo <= a.E;
    c.r0 = 0;
    c.kb = expert ? (a.K + GT_BK - 1) / GT_BK : 0;
    c.tail = (a.K - (c.kb - 1) * GT_BK + 15) >> 4;
    c.rest = 0;
  }
  c.k0 = 0;
  c.k1 = c.kb;
  if (a.ksplit > 1) {
    c.k0 = c.s * c.kb / a.ksplit;
    c.k1 = (c.s + 1) * c.kb / a.ksplit;
    if (c.s + 1 < a.ksplit) c.rest = 0;  // the last range's
  }
  return c;
}

// Arrivals on rank 0's barriers.  The producer's publishes nothing of its own
// (the copies' bytes complete the phase), so it is relaxed: a cluster-scope
// release in its place made 16,384 rows of 2,304 -> 5,760 over 64 experts take
// 905 us instead of 402.  The mender's publishes its zeros.
__device__ __forceinline__ void arrive_expect_tx_cluster(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ uint16_t to_16(float v, int kind) {
  return kind == EK_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ uint32_t pack_16(float lo, float hi, int kind) {
  return kind == EK_F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// 32 bytes to a 32-byte aligned address
__device__ __forceinline__ void store_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int OP>
__global__ void __launch_bounds__(GT_THREADS, 1)
    grouped_kernel(const __grid_constant__ GtMaps maps, const GtArgs args) {
  using Cfg = GtCfg<OP>;
  constexpr int S = GT_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * GT_A_BYTES;
  uint8_t* sS = sB + S * GT_B_BYTES;  // slices: two chunks of A, two of B each
  float* sT = reinterpret_cast<float*>(sS + Cfg::SLICES);
  uint64_t* full = reinterpret_cast<uint64_t*>(sS + Cfg::SLICES + Cfg::TURN);
  uint64_t* empty = full + S;
  uint64_t* landed = empty + S;         // a slice has landed in this CTA
  uint64_t* sfull = landed + GT_SLICES;  // it has been mended in both
  uint64_t* sempty = sfull + GT_SLICES;
  uint64_t* tfull = sempty + GT_SLICES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_plan = reinterpret_cast<int*>(sS + Cfg::SLICES + Cfg::TURN + GT_BAR_BYTES - 16);
  GtTab<OP> tab;
  tab.off = reinterpret_cast<int*>(sS + Cfg::SLICES + Cfg::TURN + GT_BAR_BYTES);
  tab.cum = tab.off + GT_MAXG + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2);    // rank 0's: an arrival from each CTA, and both CTAs' bytes
      mbar_init(smem_u32(&empty[s]), 1);   // one multicast commit
    }
    for (int b = 0; b < GT_SLICES; ++b) {
      mbar_init(smem_u32(&landed[b]), 1);  // this CTA's producer
      mbar_init(smem_u32(&sfull[b]), 2);   // rank 0's: the mender of each CTA
      mbar_init(smem_u32(&sempty[b]), 1);  // one multicast commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 8);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.A);
    prefetch_tmap(&maps.B[0]);
    if (OP == G_WGRAD) {
      prefetch_tmap(&maps.B[1]);
      prefetch_tmap(&maps.B[2]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  pdl_wait();
  if (warp == 2) gt_build<OP>(args, tab, s_plan);
  __syncthreads();
  // both CTAs' barriers are initialised before either signals the other's
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const unsigned long long tmo = args.timeout_ns;
  tab.units = s_plan[0];
  tab.whole = s_plan[1];
  tab.cuts = s_plan[2];
  const int pair = static_cast<int>(blockIdx.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------ producer (both CTAs)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued[S];
#pragma unroll
      for (int s = 0; s < S; ++s) issued[s] = -1;
      int slice = 0, slices_issued = 0;
      uint32_t slice_phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < tab.units; u += pairs_in_grid()) {
        const GtUnit c = gt_unit<OP>(args, tab, u);
        if (c.n <= 0) continue;
        const int m = c.m0 + static_cast<int>(rank) * 128;
        const int half = c.nmma / 2;  // this CTA's columns
        const int n = c.n0 + static_cast<int>(rank) * half;
        const int chunks = (half + 63) / 64;
        const uint32_t bytes = GT_A_BYTES + (OP == G_WGRAD ? chunks * 64 * GT_BK * 2 : half * GT_BK * 2);
        if (OP == G_WGRAD && c.rest > 0) {
          // the group's last, partial 16-row slice, ahead of its blocks
          if (!mbar_wait<true>(smem_u32(&sempty[slice]), slice_phase ^ 1u, tmo, abort_flag, args.status, 0x48)) break;
          const uint32_t bar = smem_u32(&landed[slice]);
          const uint32_t dst = smem_u32(sS + slice * GT_SLICE_BYTES);
          const int row = c.r0 + (c.kb > 0 ? (c.kb - 1) * GT_BK + c.tail * 16 : 0);
          mbar_arrive_expect_tx(bar, (2 + chunks) * 2048);
          tma_load_3d_pair(dst, &maps.B[1], bar, m, row, 0);
          tma_load_3d_pair(dst + 2048, &maps.B[1], bar, m + 64, row, 0);
          for (int j = 0; j < chunks; ++j) tma_load_3d_pair(dst + 4096 + j * 2048, &maps.B[2], bar, n + 64 * j, row, 0);
          ++slices_issued;
          if (++slice == GT_SLICES) {
            slice = 0;
            slice_phase ^= 1u;
          }
        }
        for (int kb = c.k0; kb < c.k1; ++kb) {
          if (!mbar_wait<true>(smem_u32(&empty[stage]), phase ^ 1u, tmo, abort_flag, args.status, 0x41)) {
            ok = false;
            break;
          }
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          arrive_expect_tx_cluster(bar, bytes);
          const uint32_t a_dst = smem_u32(sA + stage * GT_A_BYTES);
          const uint32_t b_dst = smem_u32(sB + stage * GT_B_BYTES);
          const int k0 = kb * GT_BK;
          if (OP == G_FWD) {
            tma_load_3d_pair(a_dst, &maps.A, bar, k0, m, c.e);
          } else if (OP == G_DGRAD) {
            tma_load_3d_pair(a_dst, &maps.A, bar, m, k0, c.e);
            tma_load_3d_pair(a_dst + 8192, &maps.A, bar, m + 64, k0, c.e);
          } else {
            tma_load_3d_pair(a_dst, &maps.A, bar, m, c.r0 + k0, 0);
            tma_load_3d_pair(a_dst + 8192, &maps.A, bar, m + 64, c.r0 + k0, 0);
          }
          if (OP == G_WGRAD) {
            for (int j = 0; j < chunks; ++j)
              tma_load_3d_pair(b_dst + j * 8192, &maps.B[0], bar, n + 64 * j, c.r0 + k0, 0);
          } else {
            // half rows (a multiple of 16) in boxes of 128, 64, 32 and 16 rows
            int done = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int h = 128 >> i;
              if (half & h) {
                tma_load_3d_pair(b_dst + done * 128, &maps.B[i], bar, k0, n + done, 0);
                done += h;
              }
            }
          }
          issued[stage] = static_cast<int>(phase);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (ok) {
        // the last commits of rank 0's MMAs arrive on these barriers: see
        // them all before this CTA can leave
#pragma unroll
        for (int s = 0; s < S; ++s)
          if (issued[s] >= 0 && !mbar_wait<true>(smem_u32(&empty[s]), static_cast<uint32_t>(issued[s]), tmo, abort_flag,
                                                 args.status, 0x42))
            break;
        for (int i = slices_issued > GT_SLICES ? slices_issued - GT_SLICES : 0; i < slices_issued; ++i)
          if (!mbar_wait<true>(smem_u32(&sempty[i % GT_SLICES]), (i / GT_SLICES) & 1u, tmo, abort_flag, args.status, 0x49))
            break;
      }
      if (!ok || *abort_flag) {
        // a wait ran out: give the copies in flight (they complete on barriers
        // of either CTA) time to land before the CTAs leave
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------- MMA issuer (rank 0 only)
    if (rank == 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      int slice = 0;
      uint32_t slice_phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < tab.units; u += pairs_in_grid()) {
        const GtUnit c = gt_unit<OP>(args, tab, u);
        if (c.n <= 0 || c.zero()) continue;
        if (!mbar_wait<true>(smem_u32(&tempty[acc]), acc_phase ^ 1u, tmo, abort_flag, args.status, 0x43)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
        const uint32_t idesc = args.idesc | (static_cast<uint32_t>(c.nmma >> 3) << 17);
        for (int kb = c.k0; kb < c.k1; ++kb) {
          if (!mbar_wait<true>(smem_u32(&full[stage]), phase, tmo, abort_flag, args.status, 0x44)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(sA + stage * GT_A_BYTES);
          const uint32_t b_base = smem_u32(sB + stage * GT_B_BYTES);
          const int slices = kb == c.kb - 1 ? c.tail : GT_BK / 16;
#pragma unroll
          for (int kk = 0; kk < GT_BK / 16; ++kk) {
            if (kk < slices) {
              const uint64_t ad = OP == G_FWD ? sdesc_sw128(a_base + kk * 32, 16, 1024)
                                              : sdesc_sw128(a_base + kk * 2048, 8192, 1024);
              const uint64_t bd = OP == G_WGRAD ? sdesc_sw128(b_base + kk * 2048, 8192, 1024)
                                                : sdesc_sw128(b_base + kk * 32, 16, 1024);
              umma_f16_pair(d_tmem, ad, bd, idesc, (kb > c.k0 || kk > 0) ? 1u : 0u);
            }
          }
          umma_commit_pair(smem_u32(&empty[stage]), 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (OP == G_WGRAD && c.rest > 0) {
          if (!mbar_wait<true>(smem_u32(&sfull[slice]), slice_phase, tmo, abort_flag, args.status, 0x4a)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(sS + slice * GT_SLICE_BYTES);
          umma_f16_pair(d_tmem, sdesc_sw128(a_base, 2048, 1024), sdesc_sw128(a_base + 4096, 2048, 1024), idesc,
                        c.k1 > c.k0 ? 1u : 0u);
          umma_commit_pair(smem_u32(&sempty[slice]), 0x3);
          if (++slice == GT_SLICES) {
            slice = 0;
            slice_phase ^= 1u;
          }
        }
        umma_commit_pair(smem_u32(&tfull[acc]), 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // every MMA issued must finish before either CTA frees tensor memory
      umma_commit_pair(smem_u32(drain), 0x1);
      mbar_wait<true>(smem_u32(drain), 0, ok ? tmo : 200000000ull, nullptr, args.status, 0x45);
    }
  } else if (warp == 6) {
    // ------------------------------------------------- mender (both CTAs)
    if (OP == G_WGRAD) {
      int slice = 0;
      uint32_t phase = 0;
      unsigned long long blocks = 0;  // that the producer goes through before it requests the slice
      for (int u = pair; u < tab.units; u += pairs_in_grid()) {
        const GtUnit c = gt_unit<OP>(args, tab, u);
        const int own = c.k1 - c.k0;  // after the slice
        if (c.rest == 0) {
          blocks += own;
          continue;
        }
        if (!mbar_wait(smem_u32(&landed[slice]), phase, tmo + blocks * GT_BLOCK_NS, abort_flag, args.status, 0x46)) break;
        blocks = own;
        // rows rest..15 of each chunk of 16 rows of 128 bytes
        const int words = (16 - c.rest) * 8;  // of 16 bytes
        const int chunks = (c.nmma / 2 + 63) / 64;
        for (int j = 0; j < 2 + chunks; ++j) {
          uint4* z = reinterpret_cast<uint4*>(sS + slice * GT_SLICE_BYTES + j * 2048 + c.rest * 128);
          for (int i = lane; i < words; i += 32) z[i] = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_release_cluster(mapa_shared(smem_u32(&sfull[slice]), 0));
        if (++slice == GT_SLICES) {
          slice = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;  // tensor-memory lane quadrant this warp may access
    const uint32_t tempty_cl = mapa_shared(smem_u32(&tempty[0]), 0);
    const int kind = args.out_kind;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = pair; u < tab.units; u += pairs_in_grid()) {
      const GtUnit c = gt_unit<OP>(args, tab, u);
      if (c.n <= 0) continue;
      const bool sum = !c.zero();
      if (sum &&
          !mbar_wait<true>(smem_u32(&tfull[acc]), acc_phase, tmo + (c.k1 - c.k0) * GT_BLOCK_NS, abort_flag, args.status, 0x47))
        break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
      const int row = c.m0 + static_cast<int>(rank) * 128 + q * 32;  // of the accumulator's first lane
      const int nch = (c.n + 31) / 32;
      if (OP != G_WGRAD) {
        // Y^T: lane = feature, column = row of the activations
        const int f = row + lane;
        const bool live = f < args.M;
#pragma unroll 1
        for (int ch = 0; ch < nch; ++ch) {
          uint32_t r[32];
          if (sum) {
            tmem_ld_32x32b_x32(t_row + ch * 32, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0;
          }
          const int left = c.n - ch * 32;  // columns of this chunk that are stored
          const long long base = (c.s * args.T + c.n0 + ch * 32) * args.M + f;
          if (kind == EK_F32) {
            float* p = static_cast<float*>(args.out) + base;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (live && j < left) p[static_cast<long long>(j) * args.M] = __uint_as_float(r[j]);
          } else if (args.wide) {
            // lanes 2i and 2i + 1 exchange a value: the even one stores features
            // (f, f + 1) of row j, the odd one features (f - 1, f) of row j + 1
            const bool odd = lane & 1;
            uint16_t* p = static_cast<uint16_t*>(args.out) + base + (odd ? args.M - 1 : 0);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const uint32_t got = __shfl_xor_sync(~0u, odd ? r[j] : r[j + 1], 1);
              const uint32_t v = odd ? pack_16(__uint_as_float(got), __uint_as_float(r[j + 1]), kind)
                                     : pack_16(__uint_as_float(r[j]), __uint_as_float(got), kind);
              if (live && j + (odd ? 1 : 0) < left) *reinterpret_cast<uint32_t*>(p + static_cast<long long>(j) * args.M) = v;
            }
          } else {
            uint16_t* p = static_cast<uint16_t*>(args.out) + base;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (live && j < left) p[static_cast<long long>(j) * args.M] = to_16(__uint_as_float(r[j]), kind);
          }
        }
        if (sum) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty_cl + static_cast<uint32_t>(acc * 8));
        }
      } else {
        // dW: lane = row, column = column: each lane stores along its own row,
        // whole 32-byte sectors at a time
        const long long esz = kind == EK_F32 ? 4 : 2;
        const bool live = row + lane < args.M;
        char* out = static_cast<char*>(args.out) +
                    (((static_cast<long long>(c.s) * args.E + c.e) * args.M + row + lane) * args.N + c.n0) * esz;
#pragma unroll 1
        for (int ch = 0; ch < nch; ++ch) {
          uint32_t r[32];
          if (sum) {
            tmem_ld_32x32b_x32(t_row + ch * 32, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0;
          }
          if (ch == nch - 1 && sum) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_cl + static_cast<uint32_t>(acc * 8));
          }
          char* p = out + ch * 32 * esz;
          const int left = c.n - ch * 32;
          if (args.wide && left >= 32) {
            if (kind == EK_F32) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (live) store_32(p + j * 32, r + 8 * j);
            } else {
              uint32_t h[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) h[j] = pack_16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), kind);
              if (live) {
                store_32(p, h);
                store_32(p + 32, h + 8);
              }
            }
          } else {
            // rows that are no whole sectors: turned in shared memory, then
            // stored row by row with the lanes along the row
            float* t = sT + q * 32 * 33;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j) t[lane * 33 + j] = __uint_as_float(r[j]);
            __syncwarp();
            const int rows = min(32, args.M - row);
            char* at = p - (static_cast<long long>(lane) * args.N - lane) * esz;  // the warp's first row, column `lane`
            const long long pitch = args.N * esz;
            if (args.pair_out) {  // two 16-bit columns a lane, two rows at a time
              const int r2 = lane >> 4, c2 = 2 * (lane & 15);
              char* at2 = p + (static_cast<long long>(r2 - lane) * args.N + c2) * 2;
#pragma unroll 8
              for (int i = 0; i < 32; i += 2)
                if (i + r2 < rows && c2 < left)
                  *reinterpret_cast<uint32_t*>(at2 + i * pitch) =
                      pack_16(t[(i + r2) * 33 + c2], t[(i + r2) * 33 + c2 + 1], kind);
            } else if (kind == EK_F32) {
#pragma unroll 8
              for (int i = 0; i < 32; ++i)
                if (i < rows && lane < left) *reinterpret_cast<float*>(at + i * pitch) = t[i * 33 + lane];
            } else {
#pragma unroll 8
              for (int i = 0; i < 32; ++i)
                if (i < rows && lane < left)
                  *reinterpret_cast<uint16_t*>(at + i * pitch) = to_16(t[i * 33 + lane], kind);
            }
          }
        }
      }
      if (sum && ++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // Only now: a following kernel's CTAs could not run beside this one's shared
  // memory anyway, and while they waited they would hold SMs that pairs of this
  // launch may still have to be placed on.
  pdl_trigger();
  // neither CTA leaves (or frees tensor memory) while the other may still
  // read its shared memory, write its tensor memory or arrive on its barriers
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// out[i] = the sum over s of parts[s][i], s ascending; n elements, `wide` in fours
__global__ void __launch_bounds__(256) grouped_sum_kernel(const float* parts, void* out, long long n, int splits, int kind,
                                                          int wide) {
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (wide) {
    for (; i < n / 4; i += step) {
      float4 v = reinterpret_cast<const float4*>(parts)[i];
      for (int s = 1; s < splits; ++s) {
        const float4 x = reinterpret_cast<const float4*>(parts + s * n)[i];
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
      }
      if (kind == EK_F32) reinterpret_cast<float4*>(out)[i] = v;
      else reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_16(v.x, v.y, kind), pack_16(v.z, v.w, kind));
    }
    return;
  }
  for (; i < n; i += step) {
    float v = parts[i];
    for (int s = 1; s < splits; ++s) v += parts[s * n + i];
    if (kind == EK_F32) static_cast<float*>(out)[i] = v;
    else static_cast<uint16_t*>(out)[i] = to_16(v, kind);
  }
}

// The same with the weights `a` of experts without rows left out, a warp a row:
// for calls with fewer rows than experts (20 rows, 40 experts of 999 x 1,001: 17 us
// instead of 42; where all experts have rows it is slower, 5,000 rows over 20
// experts of 1,998 x 3,002 180 us instead of 150).
__global__ void __launch_bounds__(256) grouped_pitch_rows_kernel(const PitchCopy a, const PitchCopy b, const int* offsets,
                                                                 int per_expert) {
  pdl_wait();
  pdl_trigger();
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < a.rows + b.rows;
       i += static_cast<long long>(gridDim.x) * 8) {
    const PitchCopy& p = i < a.rows ? a : b;
    const long long r = i < a.rows ? i : i - a.rows;
    if (i < a.rows) {
      const int e = static_cast<int>(r / per_expert);
      if (offsets[e + 1] <= offsets[e]) continue;
    }
#pragma unroll 4
    for (int c = (threadIdx.x & 31) * 8; c < p.cols; c += 256) pitch_word(p, r, c);
  }
}

// Ranges of every tile's reduction: more than one where the tiles are at most
// half the pairs and the reduction is long enough that a pair saves more (0.33 us
// a block) than the sums' second pass costs.  From sizes that the host knows: the
// tiles and blocks of groups of equal size.
int ksplit_of(int op, int64_t T, int64_t E, int64_t d_out, int64_t d_in, int num_sms) {
  const int64_t M = op == G_DGRAD ? d_in : d_out, m_tiles = (M + GT_BM - 1) / GT_BM;
  const int64_t groups = E < T ? E : T, share = (T + groups - 1) / groups;
  const int64_t tiles = m_tiles * (op == G_WGRAD ? E * ((d_in + GT_BN - 1) / GT_BN) : groups * ((share + GT_BN - 1) / GT_BN));
  const int64_t kb = op == G_WGRAD ? T / (GT_BK * E) : ((op == G_FWD ? d_in : d_out) + GT_BK - 1) / GT_BK;
  int64_t s = num_sms / 2 / tiles;
  if (s > 8) s = 8;
  return s > 1 && kb - kb / s >= GT_SPLIT_SAVES ? static_cast<int>(s) : 1;
}
int64_t out_elems(int op, int64_t T, int64_t E, int64_t d_out, int64_t d_in) {
  return op == G_WGRAD ? E * d_out * d_in : T * (op == G_FWD ? d_out : d_in);
}

template <int OP>
cudaError_t launch_op(const GroupedCall& g, const void* A, int64_t lda, const void* B, int64_t ldb) {
  using Cfg = GtCfg<OP>;
  auto kern = grouped_kernel<OP>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), Cfg::SMEM);
  if (e != cudaSuccess) return e;

  GtArgs a = {};
  a.out = g.C;
  a.T = g.T;
  a.M = static_cast<int>(OP == G_DGRAD ? g.d_in : g.d_out);
  a.N = static_cast<int>(g.d_in);
  a.K = static_cast<int>(OP == G_FWD ? g.d_in : g.d_out);
  a.m_tiles = (a.M + GT_BM - 1) / GT_BM;
  a.n_tiles = (a.N + GT_BN - 1) / GT_BN;
  a.n_width = ((a.N + a.n_tiles - 1) / a.n_tiles + 63) / 64 * 64;
  a.n_tiles = (a.N + a.n_width - 1) / a.n_width;
  a.ksplit = ksplit_of(OP, g.T, g.E, g.d_out, g.d_in, g.num_sms);
  const int64_t n = out_elems(OP, g.T, g.E, g.d_out, g.d_in);
  void* const result = a.ksplit > 1 ? g.parts : g.C;
  a.out = result;
  a.by_m = 1.f / static_cast<float>(a.m_tiles);
  a.by_tiles = 1.f / (static_cast<float>(a.m_tiles) * static_cast<float>(a.n_tiles));
  a.out_kind = a.ksplit > 1 ? static_cast<int>(EK_F32) : g.out_kind;
  a.idesc = idesc_f16(g.in_kind == EK_BF16, OP != G_FWD, OP == G_WGRAD, GT_BM, 0);
  a.timeout_ns = g.timeout_ns;
  a.status = g.status;
  const int esz = elem_bytes(a.out_kind);
  const uintptr_t out = reinterpret_cast<uintptr_t>(result);
  a.wide = OP == G_WGRAD ? (a.N * esz) % 32 == 0 && out % 32 == 0 : a.M % 2 == 0 && out % 4 == 0;

  a.pair_out = esz == 2 && a.N % 2 == 0 && out % 4 == 0;

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(GT_THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = g.stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;

  for (int64_t e0 = 0; e0 < g.E; e0 += GROUPED_PER_LAUNCH) {
    const int64_t ne = g.E - e0 < GROUPED_PER_LAUNCH ? g.E - e0 : GROUPED_PER_LAUNCH;
    GtMaps m;
    bool ok = true;
    const uint64_t T = g.T, di = g.d_in, dn = g.d_out;
    const uint64_t pa = static_cast<uint64_t>(lda) * 2, pb = static_cast<uint64_t>(ldb) * 2;
    if (OP == G_WGRAD) {
      ok = encode_tmap_3d(&m.A, A, g.in_kind, dn, T, 1, pa, 0, 64, 64, 128) &&
           encode_tmap_3d(&m.B[0], B, g.in_kind, di, T, 1, pb, 0, 64, 64, 128);
      ok = ok && encode_tmap_3d(&m.B[1], A, g.in_kind, dn, T, 1, pa, 0, 64, 16, 128) &&
           encode_tmap_3d(&m.B[2], B, g.in_kind, di, T, 1, pb, 0, 64, 16, 128);
      m.B[3] = m.B[0];
      a.out = static_cast<char*>(result) + e0 * g.d_out * g.d_in * esz;
    } else {
      // A: the weights [E][d_out][pitch]; B: the rows
      const char* W = static_cast<const char*>(A) + e0 * dn * pa;
      ok = encode_tmap_3d(&m.A, W, g.in_kind, di, dn, ne, pa, dn * pa, 64, OP == G_FWD ? 128 : 64, 128);
      for (int i = 0; i < 4 && ok; ++i)
        ok = encode_tmap_3d(&m.B[i], B, g.in_kind, OP == G_FWD ? di : dn, T, 1, pb, 0, 64, 128 >> i, 128);
    }
    if (!ok) return cudaErrorInvalidValue;
    a.offsets = g.offsets + e0;
    a.E = static_cast<int>(ne);
    a.first = e0 == 0;
    a.last = e0 + ne == g.E;
    // no more pairs than there can be units
    int64_t most = OP == G_WGRAD ? ne * a.m_tiles * static_cast<int64_t>(a.n_tiles)
                                 : a.m_tiles * ((ne + 2 < g.T ? ne + 2 : g.T) + g.T / GT_BN);
    most *= a.ksplit;
    int64_t pairs = g.num_sms / 2;
    if (pairs > most) pairs = most;
    if (pairs < 1) pairs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    e = cudaLaunchKernelEx(&cfg, kern, m, a);
    if (e != cudaSuccess) return e;
  }
  if (a.ksplit == 1) return cudaSuccess;
  const int wide = n % 4 == 0 && reinterpret_cast<uintptr_t>(g.C) % 16 == 0;
  int64_t blocks = ((wide ? n / 4 : n) + 255) / 256;
  if (blocks > 8 * g.num_sms) blocks = 8 * g.num_sms;
  grouped_sum_kernel<<<static_cast<unsigned>(blocks), 256, 0, g.stream>>>(static_cast<const float*>(g.parts), g.C, n,
                                                                         a.ksplit, g.out_kind, wide);
  return cudaGetLastError();
}

struct Operand {
  const void* p;
  int64_t rows, cols;
};

}  // namespace

static size_t parts_bytes(int op, int64_t T, int64_t E, int64_t d_out, int64_t d_in, int num_sms) {
  const int s = ksplit_of(op, T, E, d_out, d_in, num_sms);
  return s > 1 ? up256(static_cast<size_t>(s) * out_elems(op, T, E, d_out, d_in) * 4) : 0;
}

// The sums of split reductions, then staged copies: an operand whose rows are
// no multiple of 8 elements (or whose base is not 16-byte aligned, when `any_base`).
size_t grouped_ws_bytes(int op, int64_t T, int64_t E, int64_t d_out, int64_t d_in, bool any_base, int num_sms) {
  if (T <= 0 || E <= 0 || d_out <= 0 || d_in <= 0) return 0;
  const int64_t rows[2] = {op == G_WGRAD ? T : E * d_out, T};
  const int64_t cols[2] = {op == G_WGRAD ? d_out : d_in, op == G_DGRAD ? d_out : d_in};
  size_t n = parts_bytes(op, T, E, d_out, d_in, num_sms);
  for (int i = 0; i < 2; ++i)
    if (any_base || cols[i] % 8) n += up256(static_cast<size_t>(rows[i]) * up8(cols[i]) * 2);
  return n;
}

cudaError_t grouped_launch(const GroupedCall& call, size_t* need) {
  GroupedCall g = call;
  g.parts = g.ws;
  const Operand ops[2] = {{g.A, g.op == G_WGRAD ? g.T : g.E * g.d_out, g.op == G_WGRAD ? g.d_out : g.d_in},
                          {g.B, g.T, g.op == G_DGRAD ? g.d_out : g.d_in}};
  const void* p[2];
  int64_t pitch[2];
  size_t used = parts_bytes(g.op, g.T, g.E, g.d_out, g.d_in, g.num_sms);
  bool staged[2];
  for (int i = 0; i < 2; ++i) {
    pitch[i] = up8(ops[i].cols);
    p[i] = ops[i].p;
    staged[i] = ops[i].cols % 8 != 0 || reinterpret_cast<uintptr_t>(ops[i].p) % 16 != 0;
    if (staged[i]) {
      p[i] = static_cast<char*>(g.ws) + used;
      used += up256(static_cast<size_t>(ops[i].rows) * pitch[i] * 2);
    }
  }
  *need = used;
  if (used > 0 && (g.ws == nullptr || g.ws_bytes < used || reinterpret_cast<uintptr_t>(g.ws) % 16)) return cudaSuccess;
  *need = 0;
  if (staged[0] || staged[1]) {
    PitchCopy copy[2] = {};
    for (int i = 0; i < 2; ++i)
      if (staged[i])
        copy[i] = {static_cast<const uint16_t*>(ops[i].p), static_cast<uint16_t*>(const_cast<void*>(p[i])),
                   static_cast<long long>(ops[i].rows), static_cast<int>(ops[i].cols), static_cast<int>(pitch[i])};
    const bool sparse = g.op != G_WGRAD && staged[0] && g.T < g.E;
    int64_t grid = sparse ? (copy[0].rows + copy[1].rows + 7) / 8
                          : (copy[0].rows * (copy[0].pitch / 8) + copy[1].rows * (copy[1].pitch / 8) + 255) / 256;
    if (grid > 8 * g.num_sms) grid = 8 * g.num_sms;
    const dim3 ctas(static_cast<unsigned>(grid));
    const cudaError_t e = sparse ? launch_k(grouped_pitch_rows_kernel, ctas, dim3(256), 0, g.stream, copy[0], copy[1],
                                            g.offsets, static_cast<int>(g.d_out))
                                 : launch_k(pitch_copy_kernel, ctas, dim3(256), 0, g.stream, copy[0], copy[1]);
    if (e != cudaSuccess) return e;
  }
  switch (g.op) {
    case G_FWD: return launch_op<G_FWD>(g, p[0], pitch[0], p[1], pitch[1]);
    case G_DGRAD: return launch_op<G_DGRAD>(g, p[0], pitch[0], p[1], pitch[1]);
    default: return launch_op<G_WGRAD>(g, p[0], pitch[0], p[1], pitch[1]);
  }
}

}  // namespace tg
