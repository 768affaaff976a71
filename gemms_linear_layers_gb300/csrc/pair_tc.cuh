// pair_tc.cuh -- the skeleton of a persistent tcgen05 product on CTA pairs, for
// kernels that differ in what a unit is, what it loads and what its epilogue does.
//
// A pair computes units of 256 rows x up to 256 accumulator columns: each CTA
// loads its own 128 rows of A and its own half of B (64-deep blocks, a ring of
// P::STAGES), rank 0 issues the MMAs, each CTA's epilogue takes its 128 rows of
// one of two accumulators while the MMAs of the next unit fill the other.
// Roles of a CTA (10 warps): 0 producer (TMA), 1 MMA issuer (rank 0 of the
// pair), 2-9 epilogue: two warps a lane quadrant, which take the two halves of the
// same 64 columns, so that rows of 128 bytes leave together.  (With 32 columns a
// warp and rows of 64 bytes the epilogues of short reductions took twice as long:
// TMA moves about a row a time, and the main loop's loads wait behind the stores.)
// Every wait is bounded; the epilogue's wait for an accumulator lasts as long as a
// reduction, so its bound grows with the blocks of one.
//
// P has: Maps, Args (with units, idesc, timeout_ns, status), Unit (with kb, the
// blocks of its reduction; nmma, its columns), PARTS (1, or 2: operands in two
// 16-bit parts, a stage holds both of both, and a block is the products hi lo, lo hi and
// hi hi), STAGES, B_PART (bytes of a part of B in a stage: a CTA's half of its rows),
// EPI_BLOCKS (64-column blocks of shared memory a quadrant), State (what an epilogue warp
// keeps from unit to unit), COOPERATIVE (its units wait for others' results: every CTA has
// to be resident), and
//   idesc(args, unit)              without N and the majors
//   ready(args, unit, abort)       before the unit's copies; false: give up
//   a_mn(args, unit, kb), b_mn     is the operand of this block MN-major
//   prefetch(maps, args)           the maps of its operands
//   unit(args, u, &unit)           false: nothing to do
//   load(maps, args, unit, kb, rank, a_dst, b_dst, bar)   one block's copies
//   bytes(args, unit)              that they complete on the barrier, a CTA
//   epilogue(maps, args, unit, next, at, state, wait, release)   next: the unit after, or null
// The epilogue calls wait() before it reads the accumulator (false: give up; both
// warps of a quadrant get the same answer) and release() once it has.
#pragma once
#include <cuda.h>

#include <atomic>

#include "ptx.cuh"
#include "smem_attr.h"

namespace tg {
namespace pt {

constexpr int THREADS = 320;
constexpr int EPI_WARPS = 8;
constexpr int BK = 64;
constexpr int A_BYTES = 128 * BK * 2;  // one CTA's operand halves of a stage
constexpr int B_BYTES = 128 * BK * 2;
constexpr int BAR_BYTES = 256;
constexpr unsigned long long BLOCK_NS = 24000;  // most that a block of a reduction may take (0.2 to 1 us measured)

constexpr int BLOCK = 32 * 128;  // 32 rows x 64 columns of 16 bits
template <class P>
constexpr int smem_bytes() {
  return 1024 + P::STAGES * P::PARTS * (A_BYTES + P::B_PART) + 4 * P::EPI_BLOCKS * BLOCK + BAR_BYTES;
}

// An arrival on rank 0's barrier: it publishes nothing of its own (the copies'
// bytes complete the phase), so it is relaxed.
__device__ __forceinline__ void arrive_expect_tx_cluster(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}

// Where an epilogue warp stands.
struct EpiWarp {
  int q, h;        // lane quadrant; half of the quadrant's 64 columns
  int rank;        // CTA of the pair
  uint32_t taddr;  // tensor memory: the warp's lanes, first column of the accumulator
  uint8_t* blocks; // the quadrant's shared memory
  volatile int* abort_flag;
};
struct NoState {};
// The 64 threads of a quadrant's two warps.
__device__ __forceinline__ void quadrant_sync(int q) { asm volatile("bar.sync %0, 64;" ::"r"(q + 1) : "memory"); }
__device__ __forceinline__ bool quadrant_all(int q, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, o;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred o, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, o;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(q + 1)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ int pair_index() { return static_cast<int>(blockIdx.x >> 1); }
__device__ __forceinline__ int pair_count() { return static_cast<int>(gridDim.x >> 1); }

template <class P>
__global__ void __launch_bounds__(THREADS, 1)
    pair_kernel(const __grid_constant__ typename P::Maps maps, const __grid_constant__ typename P::Args args) {
  constexpr int S = P::STAGES;
  static_assert((2 * S + 5) * 8 + 8 <= BAR_BYTES, "barrier area");
  static_assert(smem_bytes<P>() <= 232448, "shared memory budget");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  constexpr int A_STAGE = P::PARTS * A_BYTES, B_STAGE = P::PARTS * P::B_PART;
  uint8_t* sB = sA + S * A_STAGE;
  uint8_t* sE = sB + S * B_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + 4 * P::EPI_BLOCKS * BLOCK);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2);   // rank 0's: an arrival from each CTA, and both CTAs' bytes
      mbar_init(smem_u32(&empty[s]), 1);  // one multicast commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 2 * EPI_WARPS);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    P::prefetch(maps, args);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  // both CTAs' barriers are initialised before either signals the other's
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const unsigned long long tmo = args.timeout_ns;
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------ producer (both CTAs)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued[S];
#pragma unroll
      for (int s = 0; s < S; ++s) issued[s] = -1;
      bool ok = true;
      typename P::Unit c;
      for (int u = pair_index(); ok && u < args.units; u += pair_count()) {
        if (!P::unit(args, u, c)) continue;
        if (!P::ready(args, c, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t bytes = P::bytes(args, c);
        for (int kb = 0; kb < c.kb; ++kb) {
          if (!mbar_wait<true>(smem_u32(&empty[stage]), phase ^ 1u, tmo, abort_flag, args.status, P::SITE + 1)) {
            ok = false;
            break;
          }
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          arrive_expect_tx_cluster(bar, bytes);
          P::load(maps, args, c, kb, static_cast<int>(rank), smem_u32(sA + stage * A_STAGE),
                  smem_u32(sB + stage * B_STAGE), bar);
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
                                                 args.status, P::SITE + 2))
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
      bool ok = true;
      typename P::Unit c;
      for (int u = pair_index(); ok && u < args.units; u += pair_count()) {
        if (!P::unit(args, u, c) || c.kb == 0) continue;
        if (!mbar_wait<true>(smem_u32(&tempty[acc]), acc_phase ^ 1u, tmo, abort_flag, args.status, P::SITE + 3)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
        const uint32_t idesc = P::idesc(args, c) | (static_cast<uint32_t>(c.nmma >> 3) << 17);
        for (int kb = 0; kb < c.kb; ++kb) {
          if (!mbar_wait<true>(smem_u32(&full[stage]), phase, tmo, abort_flag, args.status, P::SITE + 4)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(sA + stage * A_STAGE);
          const uint32_t b_base = smem_u32(sB + stage * B_STAGE);
          const bool a_mn = P::a_mn(args, c, kb), b_mn = P::b_mn(args, c, kb);
          const uint32_t id = idesc | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
          const uint64_t ad0 = a_mn ? sdesc_sw128(a_base, 8192, 1024) : sdesc_sw128(a_base, 16, 1024);
          const uint64_t bd0 = b_mn ? sdesc_sw128(b_base, 8192, 1024) : sdesc_sw128(b_base, 16, 1024);
          // 16 deep, in descriptor units of 16 bytes: 16 rows of an MN-major block, 32 bytes of K-major rows
          const uint64_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
#pragma unroll
          for (int p = P::PARTS == 2 ? 0 : 2; p < 3; ++p) {
            const uint64_t ad = ad0 + (p == 1 ? A_BYTES >> 4 : 0), bd = bd0 + (p == 0 ? P::B_PART >> 4 : 0);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_f16_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, id,
                            (kb > 0 || kk > 0 || (P::PARTS == 2 && p > 0)) ? 1u : 0u);
          }
          umma_commit_pair(smem_u32(&empty[stage]), 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(smem_u32(&tfull[acc]), 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // every MMA issued must finish before either CTA frees tensor memory
      umma_commit_pair(smem_u32(drain), 0x1);
      mbar_wait<true>(smem_u32(drain), 0, tmo, nullptr, args.status, P::SITE + 5);
    }
  } else {
    // ------------------------------------------------- epilogue (both CTAs)
    EpiWarp at;
    at.q = warp & 3;
    at.h = (warp - 2) >> 2;
    at.rank = static_cast<int>(rank);
    at.blocks = sE + at.q * P::EPI_BLOCKS * BLOCK;
    at.abort_flag = abort_flag;
    const uint32_t tempty_cl = mapa_shared(smem_u32(&tempty[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    typename P::State state = {};
    typename P::Unit c, next;
    for (int u = pair_index(); u < args.units; u += pair_count()) {
      if (!P::unit(args, u, c)) continue;
      const bool more = u + pair_count() < args.units && P::unit(args, u + pair_count(), next);
      at.taddr = tmem_base + (static_cast<uint32_t>(at.q * 32) << 16) + static_cast<uint32_t>(acc * 256);
      bool ok = true;
      auto wait = [&] {
        if (c.kb == 0) return true;
        ok = mbar_wait<true>(smem_u32(&tfull[acc]), acc_phase, tmo + c.kb * BLOCK_NS, abort_flag, args.status, P::SITE + 6);
        ok = quadrant_all(at.q, ok);
        tc_fence_after();
        return ok;
      };
      auto release = [&] {
        if (c.kb == 0) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_cl + static_cast<uint32_t>(acc * 8));
      };
      P::epilogue(maps, args, c, more ? &next : nullptr, at, state, wait, release);
      if (!ok) break;
      if (c.kb > 0 && ++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();
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

// Pairs that the current device holds at once, counted once a device and kernel (a
// cooperative launch of more would be refused).
template <class P>
int resident_pairs(const cudaLaunchConfig_t& cfg) {
  static std::atomic<int> known[128];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaOccupancyMaxActiveClusters(&n, pair_kernel<P>, &cfg) != cudaSuccess) return 0;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// At most `units` pairs, one a pair of SMs.
template <class P>
cudaError_t pair_launch(const typename P::Maps& maps, const typename P::Args& args, int num_sms, cudaStream_t stream) {
  auto kern = pair_kernel<P>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem_bytes<P>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes<P>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  if (P::COOPERATIVE) {
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.numAttrs = 2;
  }
  int pairs = args.units < num_sms / 2 ? args.units : num_sms / 2;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  if (P::COOPERATIVE) {
    cudaLaunchConfig_t one = cfg;  // the query takes the cluster's shape alone
    one.numAttrs = 1;
    const int most = resident_pairs<P>(one);
    if (most <= 0) return cudaErrorCooperativeLaunchTooLarge;
    if (pairs > most) pairs = most;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  }
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

// ------------------------------------------------- 32 x 64 blocks of 16 bits
// A quadrant's block in shared memory: rows of 128 bytes, 16-byte word j of row r at
// word j ^ (r % 8) (TMA's 128-byte swizzle; 1,024-byte aligned).  A lane reads and
// writes its row of its warp's half without bank conflicts.
__device__ __forceinline__ uint8_t* block_word(uint8_t* block, int row, int j) {
  return block + row * 128 + ((j ^ (row & 7)) << 4);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
  if constexpr (F16) return __half22float2(reinterpret_cast<const __half2&>(v));
  else return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(v));
}

// A lane's 32 values, rounded, into half h of its row of the block.
template <bool F16>
__device__ __forceinline__ void put_row(uint8_t* block, int lane, int h, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(block_word(block, lane, 4 * h + j)) =
        make_uint4(pack16<F16>(v[8 * j], v[8 * j + 1]), pack16<F16>(v[8 * j + 2], v[8 * j + 3]),
                   pack16<F16>(v[8 * j + 4], v[8 * j + 5]), pack16<F16>(v[8 * j + 6], v[8 * j + 7]));
}

// Half a block (32 x 32) of a matrix in global memory, in registers: word i of lane l
// is word l % 4 of row 8 i + l / 4.
struct HalfRegs {
  uint4 w[4];
};
// `rows`, `cols` of it are inside; `wide`: rows start at multiples of 16 bytes and
// cols is a multiple of 8.  What is outside reads as zero.
__device__ __forceinline__ void half_fetch(HalfRegs& r, const uint16_t* p, long long pitch, int rows, int cols, int lane,
                                           bool wide) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2), c = (lane & 3) * 8;
    r.w[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && c < cols) {
      const uint16_t* s = p + row * pitch + c;
      if (wide) {
        r.w[i] = __ldcg(reinterpret_cast<const uint4*>(s));
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = c + 2 * j < cols ? s[2 * j] : 0, hi = c + 2 * j + 1 < cols ? s[2 * j + 1] : 0;
          o[j] = lo | hi << 16;
        }
        r.w[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}
// The same straight into the block, asynchronously (words 16 bytes each; outside: zeros).
__device__ __forceinline__ void half_copy(uint8_t* block, int h, const uint16_t* p, long long pitch, int rows, int cols,
                                          int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2), c = (lane & 3) * 8;
    const bool in = row < rows && c < cols;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(block_word(block, row, 4 * h + (lane & 3)))),
                 "l"(in ? p + row * pitch + c : p), "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The warp's copies have landed, for all its lanes.
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void half_put(const HalfRegs& r, uint8_t* block, int h, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(block_word(block, 8 * i + (lane >> 2), 4 * h + (lane & 3))) = r.w[i];
}
// Half h of the block to global memory element by element, lanes along its rows: for
// rows that TMA cannot take.
__device__ __forceinline__ void half_store(uint8_t* block, int h, uint16_t* p, long long pitch, int rows, int cols, int lane) {
  __syncwarp();
#pragma unroll 4
  for (int i = 0; i < 32; ++i)
    if (i < rows && lane < cols)
      p[i * pitch + lane] = reinterpret_cast<const uint16_t*>(block_word(block, i, 4 * h + (lane >> 3)))[lane & 7];
  __syncwarp();
}

// Before a quadrant's warps write its blocks: what was stored from them has been read.
__device__ __forceinline__ void blocks_free(const EpiWarp& at, int lane) {
  if (at.h == 0 && lane == 0) bulk_wait_read<0>();
  quadrant_sync(at.q);
}
// Both have written; true in the thread that stores.
__device__ __forceinline__ bool blocks_full(const EpiWarp& at, int lane) {
  fence_async_smem();
  quadrant_sync(at.q);
  return at.h == 0 && lane == 0;
}

}  // namespace pt
}  // namespace tg
