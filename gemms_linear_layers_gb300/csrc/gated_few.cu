// gated_few.cu -- the gated feed-forward block for few rows (a token or a few dozen):
// what gated_tc.cu computes, with the weights on the M side of the MMA.
//
// With few rows a call is a stream of the weights.  A CTA takes 64 gate and the same
// 64 up rows (forward), or 128 columns of the down projection (backward), as the 128
// rows of its MMAs, and the tokens, padded to 16, as their columns; its copies fill all
// of shared memory ahead of the MMAs, 180 KB or more a CTA in flight.  Where the tiles
// leave SMs idle, a reduction is split over the CTAs of a cluster, which add each
// other's sums in rank order.
// Measured (us; in brackets the pairs of gated_tc.cu): forward, 2,304 -> 5,760, 1 row
// 11.4 (24.0; the weights alone take 7.9 at the copy rate), 16 rows 11.7 (18.8), 128
// rows 14.3 (19.0); 576 -> 1,536, 1 row 3.9 (6.2), 128 rows 5.7 (6.2).  Backward 1 row
// 8.6 (21.6), 128 rows 14.1 (18.2); of 576 -> 1,536 4.0 (6.7) and 7.7 (6.7).
#include <algorithm>
#include <type_traits>

#include "gated_act.cuh"
#include "gated_few.h"
#include "smem_attr.h"

namespace tg {
namespace {

constexpr int BK = 64;
constexpr int W_BYTES = 128 * BK * 2;
constexpr int MAX_STAGES = 12;
constexpr int BAR_BYTES = 256;
constexpr int THREADS = 384;  // warps 0-3 take the accumulator, 4 producer, 5 MMA issuer; all the epilogue

struct FewMaps {
  CUtensorMap W, X;
};
struct FewArgs {
  const uint16_t* gu_in;
  uint16_t *h, *gu;
  long long f;
  int T, kb, splits, n, stages, tmem_cols, act;
  int wide;  // G, U and the results by 16 bytes
  uint32_t idesc;
  unsigned long long timeout_ns;
  unsigned int* status;
};

template <bool F16>
__device__ __forceinline__ uint16_t round16(float v) {
  return F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
template <bool F16>
__device__ __forceinline__ float widen16(uint16_t v) {
  return F16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}

template <int V>
__device__ __forceinline__ void get(uint16_t* v, const uint16_t* p) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
  else v[0] = p[0];
}
template <int V>
__device__ __forceinline__ void put(uint16_t* p, const uint16_t* v) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
  else p[0] = v[0];
}

// v += V floats of a CTA of the cluster
template <int V>
__device__ __forceinline__ void add_remote(float* v, uint32_t addr) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 x;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                   : "r"(addr + 16 * i)
                   : "memory");
      v[4 * i] += x.x;
      v[4 * i + 1] += x.y;
      v[4 * i + 2] += x.z;
      v[4 * i + 3] += x.w;
    }
  } else {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    v[0] += x;
  }
}

template <class F>
__device__ __forceinline__ void with_act(int act, F apply) {
  switch (act) {
    case ACT_SILU: apply(std::integral_constant<int, ACT_SILU>()); break;
    case ACT_GELU: apply(std::integral_constant<int, ACT_GELU>()); break;
    case ACT_GELU_TANH: apply(std::integral_constant<int, ACT_GELU_TANH>()); break;
    default: apply(std::integral_constant<int, ACT_RELU>()); break;
  }
}

template <bool BWD, bool F16>
__global__ void __launch_bounds__(THREADS, 1) gated_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int x_bytes = a.n * BK * 2, stage_bytes = W_BYTES + x_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.stages * stage_bytes);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* done = empty + MAX_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int f0 = blockIdx.x / a.splits * (BWD ? 128 : 64);
  const int kb0 = rank * a.kb / a.splits, kb1 = (rank + 1) * a.kb / a.splits;  // this CTA's blocks
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.W);
    prefetch_tmap(&maps.X);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), a.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned long long tmo = a.timeout_ns;
  pdl_wait();

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&empty[s]), phase ^ 1u, tmo, abort_flag, a.status, 0x71)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(smem + s * stage_bytes);
        mbar_arrive_expect_tx(bar, stage_bytes);
        if (BWD) {
          tma_load_3d(dst, &maps.W, bar, f0, kb * BK, 0);
          tma_load_3d(dst + 8192, &maps.W, bar, f0 + 64, kb * BK, 0);
        } else {
          tma_load_3d(dst, &maps.W, bar, kb * BK, f0, 0);  // both planes
        }
        tma_load_3d(dst + W_BYTES, &maps.X, bar, kb * BK, 0, 0);
        if (++s == a.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok || *abort_flag) {  // copies in flight land before the CTA leaves
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------- MMA issuer
    if (elect_one()) {
      int s = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&full[s]), phase, tmo, abort_flag, a.status, 0x72)) break;
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * stage_bytes), x = w + W_BYTES;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_f16(tmem, BWD ? sdesc_sw128(w + kk * 2048, 8192, 1024) : sdesc_sw128(w + kk * 32, 16, 1024),
                   sdesc_sw128(x + kk * 32, 16, 1024), a.idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
        umma_commit(smem_u32(&empty[s]));
        if (++s == a.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      // completes when every MMA issued has: nothing of this CTA is in use after it
      umma_commit(smem_u32(done));
    }
  } else if (BWD && warp > 5) {
    // G and U on their way to L2 meanwhile: rows of 256 bytes
    const int left = static_cast<int>(a.f - f0 < 128 ? a.f - f0 : 128);
    for (int i = threadIdx.x - 192; i < a.T * 4; i += THREADS - 192) {
      const uint16_t* p = a.gu_in + static_cast<long long>(i >> 2) * 2 * a.f + (i & 1 ? a.f : 0) + f0 + (i & 2) * 32;
      if ((i & 2) * 32 < left) asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
    }
  }
  // the accumulator by tokens, [n][128], in the ring's place
  float* s = reinterpret_cast<float*>(smem);
  if (warp < 4) {
    const uint32_t row = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const bool ok = __all_sync(~0u, mbar_wait(smem_u32(done), 0, tmo + a.kb * 8000ull, abort_flag, a.status, 0x73));
    tc_fence_after();
    for (int t0 = 0; t0 < a.T && ok; t0 += 16) {
      float v[16];
      tmem_ld_32x32b_x16(row + t0, reinterpret_cast<uint32_t*>(v));
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) s[(t0 + j) * 128 + warp * 32 + lane] = v[j];
    }
  }
  __syncthreads();
  if (a.splits > 1) cluster_sync_all();
  if (!*abort_flag) {
    // ------------------------------------------------------------ epilogue
    // 8 elements a thread at a time (one where rows do not start at multiples of 16
    // bytes), BATCH of them at once; the CTAs of a cluster take them in turn
    constexpr int COLS = BWD ? 128 : 64;
    const int left = static_cast<int>(a.f - f0 < COLS ? a.f - f0 : COLS);
    auto items = [&](auto width, auto kind) {
      constexpr int V = decltype(width)::value, PER = COLS / V, BATCH = 2;
      const int step = THREADS * a.splits, all = a.T * PER;
      for (int i0 = rank * THREADS + threadIdx.x; i0 < all; i0 += BATCH * step) {
        alignas(16) uint16_t x[BATCH][V], y[BATCH][V], z[V];  // G or dG, U or dU, H
        if constexpr (BWD) {
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * step, t = i / PER, c = (i - t * PER) * V;
            if (i < all && c < left) {
              const uint16_t* p = a.gu_in + static_cast<long long>(t) * 2 * a.f + f0 + c;
              get<V>(x[k], p);
              get<V>(y[k], p + a.f);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int i = i0 + k * step, t = i / PER, c = (i - t * PER) * V;
          if (i >= all || c >= left) continue;
          float v[V], w[V];  // dH; or G and U
          const float* p = s + t * 128 + c;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            v[e] = w[e] = 0.f;
            if (a.splits == 1) {
              v[e] = p[e];
              if (!BWD) w[e] = p[64 + e];
            }
          }
          for (int r = 0; r < a.splits && a.splits > 1; ++r) {
            const uint32_t q = mapa_shared(smem_u32(p), r);
            add_remote<V>(v, q);
            if (!BWD) add_remote<V>(w, q + 256);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if constexpr (BWD) {
              const float g = widen16<F16>(x[k][e]), u = widen16<F16>(y[k][e]);
              float value;
              const float slope = activation_grad<decltype(kind)::value>(g, &value);
              x[k][e] = round16<F16>(v[e] * u * slope);
              y[k][e] = round16<F16>(v[e] * value);
              z[e] = round16<F16>(value * u);
            } else {
              x[k][e] = round16<F16>(v[e]);
              y[k][e] = round16<F16>(w[e]);
              z[e] = round16<F16>(activation<decltype(kind)::value>(v[e]) * w[e]);
            }
          }
          const long long at = static_cast<long long>(t) * a.f + f0 + c, gu = at + static_cast<long long>(t) * a.f;
          if (a.gu) {
            put<V>(a.gu + gu, x[k]);
            put<V>(a.gu + gu + a.f, y[k]);
          }
          if (a.h) put<V>(a.h + at, z);
        }
      }
    };
    with_act(a.act, [&](auto kind) {
      if (a.wide) items(std::integral_constant<int, 8>(), kind);
      else items(std::integral_constant<int, 1>(), kind);
    });
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (a.splits > 1) cluster_sync_all();  // the others have read this CTA's sums
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }
}

template <bool BWD, bool F16>
cudaError_t launch_few(const GatedFew& g) {
  FewMaps m = {};
  FewArgs a = {};
  a.gu_in = static_cast<const uint16_t*>(g.GU);
  a.h = static_cast<uint16_t*>(g.H);
  a.gu = static_cast<uint16_t*>(g.out);
  a.f = g.f;
  a.T = static_cast<int>(g.T);
  a.kb = static_cast<int>((g.d + BK - 1) / BK);
  a.n = (a.T + 15) / 16 * 16;
  a.tmem_cols = a.n <= 32 ? 32 : a.n <= 64 ? 64 : 128;
  a.act = g.act;
  a.idesc = idesc_f16(!F16, BWD, false, 128, a.n);
  a.wide = g.f % 8 == 0;
  for (const void* p : {g.GU, static_cast<const void*>(g.H), static_cast<const void*>(g.out)})
    a.wide = a.wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  a.timeout_ns = g.timeout_ns;
  a.status = g.status;
  const int stage = W_BYTES + a.n * BK * 2;
  a.stages = (232448 - 1024 - BAR_BYTES) / stage;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  const int smem = 1024 + a.stages * stage + BAR_BYTES;  // the epilogue's n x 512 bytes are less than the ring
  const uint64_t pw = static_cast<uint64_t>(g.pitch_w) * 2, px = static_cast<uint64_t>(g.pitch_x) * 2;
  const int kind = F16 ? EK_F16 : EK_BF16;
  bool ok = encode_tmap_3d(&m.X, g.A, kind, g.d, g.T, 1, px, 0, BK, a.n, 128);
  if (BWD) {
    ok = ok && encode_tmap_3d(&m.W, g.W, kind, g.f, g.d, 1, pw, 0, 64, BK, 128);
  } else {
    const uint64_t dims[3] = {static_cast<uint64_t>(g.d), static_cast<uint64_t>(g.f), 2};
    const uint64_t strides[2] = {pw, g.f * pw};
    const uint32_t box[3] = {BK, 64, 2};
    ok = ok && encode_tmap_nd(&m.W, g.W, kind, 3, dims, strides, box, 128);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto kern = gated_few_kernel<BWD, F16>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t per = BWD ? 128 : 64, tiles = (g.f + per - 1) / per;
  // Ranges of at least 6 blocks for SMs that the tiles leave idle.  At most 4: more than
  // a GPC's SMs hold of larger clusters wait for a second round (128 rows, 2,304 -> 1,000:
  // clusters of 6 and 8 21 us, of 4 10).
  int64_t splits = std::min<int64_t>(std::min<int64_t>(g.num_sms / tiles, a.kb / 6), 4);
  a.splits = static_cast<int>(splits < 1 ? 1 : splits);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = g.stream;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, m, a);
}

}  // namespace

cudaError_t gated_few_launch(const GatedFew& g) {
  if (g.in_kind == EK_F16) return g.bwd ? launch_few<true, true>(g) : launch_few<false, true>(g);
  return g.bwd ? launch_few<true, false>(g) : launch_few<false, false>(g);
}

}  // namespace tg
