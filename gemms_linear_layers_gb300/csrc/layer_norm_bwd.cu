// layer_norm_bwd.cu -- backward of layer_norm_fwd.cu, for dY (means over the row):
//   n  = (X - mean) rstd,  q = dY w
//   dX = rstd (q - mean(q) - n mean(q n)) + dR
//   dw = sum_t dY n,  db = sum_t dY
// FP32 arithmetic, every output rounded once.  Bound by HBM: 2 values (3 with
// dR) read and one written an element, in one pass with one exchange a row: both
// means are sums of values that a thread has at hand.  The column sums build up
// in registers (in shared memory with 4 groups a thread); the teams of a CTA
// are added in shared memory, the CTAs by a second launch, all in a fixed order.
#include "layer_norm.h"
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

// Groups a thread: 1 while an SM's registers hold a row's threads, 3 beyond (48
// column sums in registers), then 4 (sums in shared memory).  One CTA an SM
// (few partial sums): its threads.
constexpr int LNB_MANY = 3, LNB_WIDEST = 4;
constexpr int lnb_threads(int vpt) { return vpt > 1 ? 512 : 864; }
constexpr int LNB_DEPTH = 2;  // rows in the ring

struct LnbArgs {
  const void *X, *w, *dY, *dR;
  const float *mean, *rstd;
  void* dX;
  float* part;  // [CTA][2][d]: dw, db
  long long T;
  int d, team, teams, classes;
};

// Sums of two values over the team; every thread gets them, added in the same order.
__device__ __forceinline__ float2 team_sum2(float2 v, float2* slot, int which, int team_id, int team, int t) {
  auto warp_sum = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(~0u, v.x, o);
      v.y += __shfl_xor_sync(~0u, v.y, o);
    }
  };
  warp_sum();
  const int warps = team >> 5;
  if (warps == 1) return v;
  float2* s = slot + which * 32;
  if ((t & 31) == 0) s[t >> 5] = v;
  team_sync(team_id, team);
  v = (t & 31) < warps ? s[t & 31] : both(0.f);
  warp_sum();
  return v;
}

template <typename IN, int VPT, int FEED>
__global__ void __launch_bounds__(lnb_threads(VPT), 1) layer_norm_bwd_kernel(const LnbArgs a) {
  constexpr bool RING = FEED == FEED_RING || FEED == FEED_SHIFT;
  constexpr int D = LNB_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];  // the ring, then the column sums
  __shared__ float2 slots[2][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  float2* slot = slots[0] + team_id * (a.team >> 5);
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool res = a.dR != nullptr;
  const int group_words = (res ? 3 : 2) * Pack<IN>::WORDS;
  const Ring ring = ring_of(ring_smem, VPT * group_words);
  if (RING) ring_clear(ring, VPT * group_words, D);
  pdl_wait();
  pdl_trigger();
  // rows: those congruent to `cls` modulo a.classes, dealt to the teams of the CTAs with that class in turn
  const int cls = blockIdx.x % a.classes;
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  const long long row0 = cls + static_cast<long long>(a.classes) * ((blockIdx.x / a.classes) * a.teams + team_id);
  const int shift = FEED == FEED_SHIFT ? static_cast<int>((static_cast<long long>(cls) * d) & 7) : 0;
  auto fetch = [&](long long row, int stage) {
    if (row < a.T) {
      const long long rest = (a.T - row) * d;
      const int left = rest < (1 << 30) ? static_cast<int>(rest) : 1 << 30;
      int w = 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
        ring_copy<IN, FEED>(ring, stage, w, a.X, row, c, d, left);
        ring_copy<IN, FEED>(ring, stage, w, a.dY, row, c, d, left);
        if (res) ring_copy<IN, FEED>(ring, stage, w, a.dR, row, c, d, left);
      }
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(row0 + i * step, i);
  }
  // 4 groups a thread (one team a CTA): column sum k of the thread's group v, half i at (((k * VPT + v) * 2 + i) * team + t)
  constexpr bool IN_SMEM = VPT == LNB_WIDEST;
  const int ring_bytes = RING ? D * static_cast<int>(ring.stage) : 0;
  float4* accs = reinterpret_cast<float4*>(ring_smem + ring_bytes) + t;
  auto at = [&](int k, int v, int i) -> float4& { return accs[((k * VPT + v) * 2 + i) * a.team]; };
  auto add8 = [&](int k, int v, const float2* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 f = at(k, v, i);
      f.x += x[2 * i].x;
      f.y += x[2 * i].y;
      f.z += x[2 * i + 1].x;
      f.w += x[2 * i + 1].y;
      at(k, v, i) = f;
    }
  };
  if (IN_SMEM) {
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) at(k, v, 0) = at(k, v, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // FEED_SHIFT: w beside the ring
  IN* sw = reinterpret_cast<IN*>(ring_smem + ring_bytes);
  const int groups = VPT * a.team;
  if (FEED == FEED_SHIFT) {
    lay_shifted<IN>(sw, 0, a.w, groups, d, shift);
    __syncthreads();
  }
  constexpr int KEPT = IN_SMEM ? 1 : VPT;
  float2 acc_w[KEPT][4] = {}, acc_b[KEPT][4] = {};
  int which = 0, stage = 0;
  // a row's scalars are loaded a row ahead too
  float mean_next = 0.f, rstd_next = 0.f;
  auto scalars = [&](long long row) {
    if (row < a.T) {
      mean_next = a.mean[row];
      rstd_next = a.rstd[row];
    }
  };
  scalars(row0);
  for (long long row = row0; row < a.T; row += step) {
    const float2 centre = both(-mean_next), rstd = both(rstd_next);
    scalars(row + step);
    if (RING) {
      fetch(row + (D - 1) * step, stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<IN>(a.X, row + step, d, t, a.team);
      prefetch_row<IN>(a.dY, row + step, d, t, a.team);
      if (res) prefetch_row<IN>(a.dR, row + step, d, t, a.team);
    }
    // X (and dR) are taken twice: all of it kept between the two would spill
    auto take = [&](const void* from, int v, int k, const Cols<FEED>& c) {
      if constexpr (RING) {
        int w = v * group_words + k * Pack<IN>::WORDS;
        return ring_read<IN, FEED>(ring, stage, w, c, d);
      } else {
        return load8<IN, FEED>(from, row, c, d);
      }
    };
    float2 s1 = both(0.f), s2 = both(0.f);
    float2 q[VPT][4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> x = take(a.X, v, 0, c), g = take(a.dY, v, 1, c);
      Pack<IN> w;
      if constexpr (FEED == FEED_SHIFT) w = read_shifted<IN>(sw, 0, groups, v * a.team + t);
      else w = load8<IN, FEED>(a.w, 0, c, d);
      float2 gy[4], gn[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 n = mul2(add2(two(x, j), centre), rstd);
        gy[j] = two(g, j);
        gn[j] = mul2(gy[j], n);
        q[v][j] = mul2(gy[j], two(w, j));
        s1 = add2(s1, q[v][j]);
        s2 = fma2(q[v][j], n, s2);
        if constexpr (!IN_SMEM) {
          acc_w[v][j] = add2(acc_w[v][j], gn[j]);
          acc_b[v][j] = add2(acc_b[v][j], gy[j]);
        }
      }
      if (IN_SMEM) {
        add8(0, v, gn);
        add8(1, v, gy);
      }
    }
    const float2 sum = team_sum2(make_float2(s1.x + s1.y, s2.x + s2.y), slot, which, team_id, a.team, t);
    which ^= 1;
    // dX = rstd q + (-rstd mean(q)) + n (-rstd mean(q n))
    const float2 m1 = both(-rstd.x * (sum.x * inv_d)), m2 = both(-rstd.x * (sum.y * inv_d));
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> x = take(a.X, v, 0, c);
      float2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 n = mul2(add2(two(x, j), centre), rstd);
        o[j] = fma2(rstd, q[v][j], fma2(n, m2, m1));
      }
      if (res) {
        const Pack<IN> r = take(a.dR, v, 2, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = add2(o[j], two(r, j));
      }
      store8<IN, FEED>(a.dX, row, c, d, o);
    }
    stage = stage + 1 < D ? stage + 1 : 0;
  }
  if (RING) ring_wait<0>();
  float* out = a.part + static_cast<long long>(blockIdx.x) * 2 * d;
  if (IN_SMEM) {
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 f = at(k, v, i);
          if (c[4 * i] < d) out[k * d + c[4 * i]] = f.x;
          if (c[4 * i + 1] < d) out[k * d + c[4 * i + 1]] = f.y;
          if (c[4 * i + 2] < d) out[k * d + c[4 * i + 2]] = f.z;
          if (c[4 * i + 3] < d) out[k * d + c[4 * i + 3]] = f.w;
        }
      }
    return;
  }
  // the CTA's column sums: the teams one after the other, in the ring's place
  float* col = reinterpret_cast<float*>(ring_smem);
  for (int k = 0; k < a.teams; ++k) {
    __syncthreads();
    if (team_id == k) {
#pragma unroll
      for (int v = 0; v < KEPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c[j] >= 0 && c[j] < d) {
            float* p = col + c[j];
            p[0] = (k ? p[0] : 0.f) + (j & 1 ? acc_w[v][j / 2].y : acc_w[v][j / 2].x);
            p[d] = (k ? p[d] : 0.f) + (j & 1 ? acc_b[v][j / 2].y : acc_b[v][j / 2].x);
          }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) out[i] = col[i];
}

Geo lnb_geometry(int64_t T, int64_t d, bool shift, int sms) {
  int vpt = 1;
  for (const int v : {LNB_MANY, LNB_WIDEST})
    if (team_of(width_of(d, shift), vpt) > lnb_threads(vpt)) vpt = v;
  Geo g = geometry(T, d, shift, sms, vpt, lnb_threads(vpt), 1);
  if (vpt == LNB_WIDEST) {  // one row at a time
    g.teams = 1;
    g.ctas = static_cast<int>(T < sms ? T : sms);
  }
  return g;
}
// Bytes of shared memory: the ring and FEED_SHIFT's weights, and the column
// sums, beside those (4 groups a thread) or in their place.
template <typename IN>
int lnb_smem(const LayerNorm& n, const Geo& g, int feed) {
  const int words = g.vpt * (n.dR ? 3 : 2) * Pack<IN>::WORDS;
  int rows = feed == FEED_RING || feed == FEED_SHIFT ? LNB_DEPTH * words * g.team * g.teams * 16 : 0;
  if (feed == FEED_SHIFT) rows += g.vpt * g.team * 8 * static_cast<int>(sizeof(IN));
  const int sums = static_cast<int>(g.vpt == LNB_WIDEST ? 2 * g.vpt * g.team * 32 : 2 * n.d * 4);
  return g.vpt == LNB_WIDEST ? rows + sums : rows > sums ? rows : sums;
}

template <typename IN, int VPT, int FEED>
cudaError_t lnb_one(const LayerNorm& n, const Geo& g) {
  const LnbArgs a = {n.X, n.w, n.dY, n.dR, n.mean, n.rstd, n.dX, n.ws, n.T, static_cast<int>(n.d), g.team, g.teams, g.classes};
  *n.rows = FEED_NAMES[FEED];
  auto kern = layer_norm_bwd_kernel<IN, VPT, FEED>;
  const int smem = lnb_smem<IN>(n, g, FEED);
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  e = launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
  if (e != cudaSuccess) return e;
  const int sums = n.db ? 2 : 1;
  return launch_k(norm_cols_kernel, dim3(static_cast<unsigned>((sums * n.d + 31) / 32)), dim3(1024), 0, n.stream,
                  static_cast<const float*>(n.ws), g.ctas, static_cast<int>(n.d), 2, sums, n.dw, n.db, n.db, n.out_kind);
}
template <typename IN>
cudaError_t lnb_types(const LayerNorm& n) {
  const bool words = aligned16({n.X, n.w, n.dY, n.dR, n.dX});
  // through the ring, with fewer rows at once (no fewer CTAs) where they do not fit
  auto fit = [&](bool shift, int feed, Geo* g) {
    *g = lnb_geometry(n.T, n.d, shift, n.num_sms);
    while (g->teams > 1 && lnb_smem<IN>(n, *g, feed) > SMEM_BYTES) --g->teams;
    return words && (n.d % 8 != 0) == shift && g->vpt != LNB_WIDEST && lnb_smem<IN>(n, *g, feed) <= SMEM_BYTES;
  };
  Geo g;
  if (fit(true, FEED_SHIFT, &g))
    return g.vpt == 1 ? lnb_one<IN, 1, FEED_SHIFT>(n, g) : lnb_one<IN, LNB_MANY, FEED_SHIFT>(n, g);
  if (fit(false, FEED_RING, &g))
    return g.vpt == 1 ? lnb_one<IN, 1, FEED_RING>(n, g) : lnb_one<IN, LNB_MANY, FEED_RING>(n, g);
  g = lnb_geometry(n.T, n.d, false, n.num_sms);
  // aligned rows of up to 3 groups a thread always fit the ring, but FP32 ones with dR
  const bool vec = words && n.d % 8 == 0;
  if (g.vpt == 1) return lnb_one<IN, 1, FEED_SCALAR>(n, g);
  if (g.vpt == LNB_MANY) {
    if constexpr (sizeof(IN) == 4) {
      if (vec) return lnb_one<IN, LNB_MANY, FEED_VEC>(n, g);
    }
    return lnb_one<IN, LNB_MANY, FEED_SCALAR>(n, g);
  }
  return vec ? lnb_one<IN, LNB_WIDEST, FEED_VEC>(n, g) : lnb_one<IN, LNB_WIDEST, FEED_SCALAR>(n, g);
}

}  // namespace

size_t layer_norm_bwd_ws_bytes(int64_t T, int64_t d, int num_sms) {
  if (T <= 0 || d <= 0) return 0;
  return static_cast<size_t>((T < num_sms ? T : num_sms) + 7) * 2 * d * 4;  // of each CTA (whole rounds of up to 8 classes)
}

cudaError_t layer_norm_bwd_launch(const LayerNorm& n) {
  switch (n.in_kind) {
    case EK_BF16: return lnb_types<__nv_bfloat16>(n);
    case EK_F16: return lnb_types<__half>(n);
    default: return lnb_types<float>(n);
  }
}

}  // namespace tg
