// layer_norm_bwd.cu -- backward of layer_norm_fwd.cu, for dY (means over the row):
//   n  = (X - mean) rstd,  q = dY w
//   dX = rstd (q - mean(q) - n mean(q n)) + dR
//   dw = sum_t dY n,  db = sum_t dY
// FP32 arithmetic, every output rounded once.  Bound by HBM: 2 values (3 with
// dR) read and one written an element, in one pass with one exchange a row: both
// means are sums of values that a thread has at hand.  The column sums build up
// in registers (in shared memory with 4 groups a thread); the teams of a CTA
// are added in shared memory, the CTAs by a second launch, all in a fixed order.
// Measured: 8,192 x 2,304 bf16 with dR 34 us, 4.4 TB/s, without 31 us; 65,536 x 2,304
// 179 us, 5.1 TB/s; 16,384 x 576 21 us; 2,047 x 576 FP32 10.4 us (4 of them the second
// launch); 8,192 x 2,301 with dR 46 us.
#include "layer_norm.h"
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

// Groups a thread: 1 while an SM's registers hold a row's threads, 3 beyond (48
// column sums in registers), then 4 (sums in shared memory).  One CTA an SM
// (few partial sums): its threads (864 of 72 registers spill: 8,192 x 2,304 with dR 42 us).
constexpr int LNB_MANY = 3, LNB_WIDEST = 4;
constexpr int lnb_threads(int vpt) { return vpt > 1 ? 512 : 640; }
constexpr int LNB_DEPTH = 2;  // stages of the ring

struct LnbArgs {
  const void *X, *w, *dY, *dR;
  const float *mean, *rstd;
  void* dX;
  float* part;  // [CTA][2][d]: dw, db
  long long T;
  int d, team, teams, classes;
};

// Sums of four values over the team; every thread gets them, added in the same order.
__device__ __forceinline__ float4 team_sum4(float4 v, float4* slot, int which, int team_id, int team, int t) {
  auto warp_sum = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(~0u, v.x, o);
      v.y += __shfl_xor_sync(~0u, v.y, o);
      v.z += __shfl_xor_sync(~0u, v.z, o);
      v.w += __shfl_xor_sync(~0u, v.w, o);
    }
  };
  warp_sum();
  const int warps = team >> 5;
  if (warps == 1) return v;
  float4* s = slot + which * 32;
  if ((t & 31) == 0) s[t >> 5] = v;
  team_sync(team_id, team);
  v = (t & 31) < warps ? s[t & 31] : make_float4(0.f, 0.f, 0.f, 0.f);
  warp_sum();
  return v;
}

// ROWS rows of a team at a time: their sums are exchanged together, and w is taken once for all of them.
template <typename IN, int VPT, int FEED, int ROWS>
__global__ void __launch_bounds__(lnb_threads(VPT), 1) layer_norm_bwd_kernel(const LnbArgs a) {
  constexpr bool RING = FEED == FEED_RING || FEED == FEED_SHIFT;
  constexpr int D = LNB_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];  // the ring, then the column sums
  __shared__ float4 slots[2][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  float4* slot = slots[0] + team_id * (a.team >> 5);
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool res = a.dR != nullptr;
  const int group_words = (res ? 3 : 2) * Pack<IN>::WORDS;
  const Ring ring = ring_of(ring_smem, ROWS * VPT * group_words);
  if (RING) ring_clear(ring, ROWS * VPT * group_words, D);
  pdl_wait();
  pdl_trigger();
  // rows: those congruent to `cls` modulo a.classes, dealt to the teams of the CTAs with that class in turn
  const int cls = blockIdx.x % a.classes;
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  const long long row0 = cls + static_cast<long long>(a.classes) * ((blockIdx.x / a.classes) * a.teams + team_id);
  const int shift = FEED == FEED_SHIFT ? static_cast<int>((static_cast<long long>(cls) * d) & 7) : 0;
  // offsets of the row to ask for and of the row at work move on by additions
  const long long stride = step * d;
  long long ask = row0 * d, ask_row = row0;
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r, ask_row += step, ask += stride) {
      if (ask_row < a.T) {
        int left = 1 << 30;
        if (FEED == FEED_SHIFT && (a.T - ask_row) * d < left) left = static_cast<int>((a.T - ask_row) * d);
        int w = r * VPT * group_words;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const Cols<FEED> c(v, t, a.team, d, shift);
          ring_copy<IN, FEED>(ring, stage, w, static_cast<const IN*>(a.X) + ask, 0, c, d, left);
          ring_copy<IN, FEED>(ring, stage, w, static_cast<const IN*>(a.dY) + ask, 0, c, d, left);
          if (res) ring_copy<IN, FEED>(ring, stage, w, static_cast<const IN*>(a.dR) + ask, 0, c, d, left);
        }
      }
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(i);
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
  // a row's scalars are loaded a round ahead too; a row past the last has rstd 0 and adds nothing
  float mean_next[ROWS], rstd_next[ROWS];
  auto scalars = [&](long long row) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r, row += step) {
      mean_next[r] = row < a.T ? a.mean[row] : 0.f;
      rstd_next[r] = row < a.T ? a.rstd[row] : 0.f;
    }
  };
  scalars(row0);
  // w stays in registers where a thread has one group
  constexpr bool KEEP = VPT == 1 && FEED == FEED_RING && sizeof(IN) == 2;
  Pack<IN> kept_w;
  if (KEEP) kept_w = load8<IN, FEED>(a.w, 0, Cols<FEED>(0, t, a.team, d, shift), d);
  long long at_row = row0 * d;
  for (long long row = row0; row < a.T; row += ROWS * step, at_row += ROWS * stride) {
    float mean[ROWS], rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      mean[r] = mean_next[r];
      rstd[r] = rstd_next[r];
    }
    scalars(row + ROWS * step);
    if (RING) {
      fetch(stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<IN>(a.X, row + step, d, t, a.team);
      prefetch_row<IN>(a.dY, row + step, d, t, a.team);
      if (res) prefetch_row<IN>(a.dR, row + step, d, t, a.team);
    }
    // X (and dR) are taken twice: all of it kept between the two would spill
    auto take = [&](const void* from, int r, int v, int k, const Cols<FEED>& c) {
      if constexpr (RING) {
        int w = (r * VPT + v) * group_words + k * Pack<IN>::WORDS;
        return ring_read<IN, FEED>(ring, stage, w, c, d);
      } else {
        return load8<IN, FEED>(static_cast<const IN*>(from) + at_row, 0, c, d);
      }
    };
    auto live = [&](int r) { return r == 0 || row + r * step < a.T; };
    float2 s1[ROWS], s2[ROWS];  // of q, and of q (X - mean)
    float2 q[ROWS][VPT][4];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s1[r] = s2[r] = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      Pack<IN> w;
      if constexpr (KEEP) w = kept_w;
      else if constexpr (FEED == FEED_SHIFT) w = read_shifted<IN>(sw, 0, groups, v * a.team + t);
      else w = load8<IN, FEED>(a.w, 0, c, d);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const Pack<IN> x = take(a.X, r, v, 0, c);
        Pack<IN> g = take(a.dY, r, v, 1, c);
        if (!live(r)) g = zeros<IN>();  // the ring holds an older row there
        float2 gy[4], gn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 xc = add2(two(x, j), both(-mean[r]));
          gy[j] = two(g, j);
          q[r][v][j] = mul2(gy[j], two(w, j));
          s1[r] = add2(s1[r], q[r][v][j]);
          s2[r] = fma2(q[r][v][j], xc, s2[r]);
          gn[j] = mul2(gy[j], both(rstd[r]));
          if constexpr (!IN_SMEM) {
            acc_w[v][j] = fma2(gn[j], xc, acc_w[v][j]);
            acc_b[v][j] = add2(acc_b[v][j], gy[j]);
          } else {
            gn[j] = mul2(gn[j], xc);
          }
        }
        if (IN_SMEM) {
          add8(0, v, gn);
          add8(1, v, gy);
        }
      }
    }
    const float4 sum = team_sum4(make_float4(s1[0].x + s1[0].y, s2[0].x + s2[0].y, ROWS > 1 ? s1[ROWS - 1].x + s1[ROWS - 1].y : 0.f,
                                             ROWS > 1 ? s2[ROWS - 1].x + s2[ROWS - 1].y : 0.f),
                                 slot, which, team_id, a.team, t);
    which ^= 1;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (!live(r)) continue;
      // dX = rstd q + (-rstd mean(q)) + (X - mean) (-rstd^2 mean(q n))
      const float2 k = both(rstd[r]), m1 = both(-rstd[r] * ((r ? sum.z : sum.x) * inv_d));
      const float2 m2 = both(-rstd[r] * (rstd[r] * (rstd[r] * ((r ? sum.w : sum.y) * inv_d))));
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
        const Pack<IN> x = take(a.X, r, v, 0, c);
        float2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = fma2(k, q[r][v][j], fma2(add2(two(x, j), both(-mean[r])), m2, m1));
        if (res) {
          const Pack<IN> p = take(a.dR, r, v, 2, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = add2(o[j], two(p, j));
        }
        store8<IN, FEED>(static_cast<IN*>(a.dX) + at_row + r * stride, 0, c, d, o);
      }
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
  // the CTA's column sums: those of each team side by side in the ring's place, [teams][2][d], added in order
  float* col = reinterpret_cast<float*>(ring_smem);
  __syncthreads();
#pragma unroll
  for (int v = 0; v < KEPT; ++v) {
    const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c[j] >= 0 && c[j] < d) {
        float* p = col + 2 * team_id * d + c[j];
        p[0] = j & 1 ? acc_w[v][j / 2].y : acc_w[v][j / 2].x;
        p[d] = j & 1 ? acc_b[v][j / 2].y : acc_b[v][j / 2].x;
      }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
    float v = col[i];
    for (int k = 1; k < a.teams; ++k) v += col[2 * k * d + i];
    out[i] = v;
  }
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
int lnb_smem(const LayerNorm& n, const Geo& g, int feed, int at_once) {
  const int words = at_once * g.vpt * (n.dR ? 3 : 2) * Pack<IN>::WORDS;
  int rows = feed == FEED_RING || feed == FEED_SHIFT ? LNB_DEPTH * words * g.team * g.teams * 16 : 0;
  if (feed == FEED_SHIFT) rows += g.vpt * g.team * 8 * static_cast<int>(sizeof(IN));
  const int sums = static_cast<int>(g.vpt == LNB_WIDEST ? 2 * g.vpt * g.team * 32 : g.teams * 2 * n.d * 4);
  return g.vpt == LNB_WIDEST ? rows + sums : rows > sums ? rows : sums;
}

template <typename IN, int VPT, int FEED, int ROWS>
cudaError_t lnb_one(const LayerNorm& n, const Geo& g) {
  const LnbArgs a = {n.X, n.w, n.dY, n.dR, n.mean, n.rstd, n.dX, n.ws, n.T, static_cast<int>(n.d), g.team, g.teams, g.classes};
  *n.rows = FEED_NAMES[FEED];
  auto kern = layer_norm_bwd_kernel<IN, VPT, FEED, ROWS>;
  const int smem = lnb_smem<IN>(n, g, FEED, ROWS);
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
  // through the ring, with fewer teams (no fewer CTAs) where their rows do not fit
  auto fit = [&](bool shift, int feed, int at_once, Geo* g) {
    *g = lnb_geometry(n.T, n.d, shift, n.num_sms);
    while (g->teams > 1 && lnb_smem<IN>(n, *g, feed, at_once) > SMEM_BYTES) --g->teams;
    return words && (n.d % 8 != 0) == shift && g->vpt != LNB_WIDEST && lnb_smem<IN>(n, *g, feed, at_once) <= SMEM_BYTES;
  };
  Geo g;
  const bool shift = n.d % 8 != 0;
  // two rows at a time where a team has several
  if (fit(shift, shift ? FEED_SHIFT : FEED_RING, 2, &g) && g.vpt == 1 && n.T >= 4 * static_cast<int64_t>(g.ctas) * g.teams)
    return shift ? lnb_one<IN, 1, FEED_SHIFT, 2>(n, g) : lnb_one<IN, 1, FEED_RING, 2>(n, g);
  if (shift && fit(true, FEED_SHIFT, 1, &g))
    return g.vpt == 1 ? lnb_one<IN, 1, FEED_SHIFT, 1>(n, g) : lnb_one<IN, LNB_MANY, FEED_SHIFT, 1>(n, g);
  if (!shift && fit(false, FEED_RING, 1, &g))
    return g.vpt == 1 ? lnb_one<IN, 1, FEED_RING, 1>(n, g) : lnb_one<IN, LNB_MANY, FEED_RING, 1>(n, g);
  g = lnb_geometry(n.T, n.d, false, n.num_sms);
  // aligned rows of up to 3 groups a thread always fit the ring, but FP32 ones with dR
  const bool vec = words && n.d % 8 == 0;
  if (g.vpt == 1) return lnb_one<IN, 1, FEED_SCALAR, 1>(n, g);
  if (g.vpt == LNB_MANY) {
    if constexpr (sizeof(IN) == 4) {
      if (vec) return lnb_one<IN, LNB_MANY, FEED_VEC, 1>(n, g);
    }
    return lnb_one<IN, LNB_MANY, FEED_SCALAR, 1>(n, g);
  }
  return vec ? lnb_one<IN, LNB_WIDEST, FEED_VEC, 1>(n, g) : lnb_one<IN, LNB_WIDEST, FEED_SCALAR, 1>(n, g);
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
