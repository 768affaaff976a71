// layer_norm_fwd.cu -- layer norm over the rows of X:
//   mean = sum_c X / d,  rstd = (sum_c (X - mean)^2 / d + eps)^-1/2
//   Y    = (X - mean) rstd w + b
// FP32 arithmetic, every output rounded once.  The squares are taken of
// distances from a mean, never of X itself, so a row far from zero keeps its
// variance; a row still costs one exchange between its warps: each warp takes
// its own columns' mean and the squares around that, and the warps' pairs (of
// n_w columns, mean m_w, squares M_w) join as
//   mean = sum n_w m_w / d,   M = sum (M_w + n_w (m_w - mean)^2).
// Bound by HBM: a value read and a value written an element.
#include "layer_norm.h"
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

constexpr int LNF_MANY = 3;   // groups of eight columns a thread where rows are many or wide
constexpr int lnf_threads(int vpt) { return vpt == 1 ? 1024 : 768; }
constexpr int LNF_CTA = 384;  // a CTA of several rows
constexpr int LNF_DEPTH = 3;  // rows in the ring

struct LnfArgs {
  const void *X, *w, *b;
  void* Y;
  float *mean, *rstd;
  long long T;
  int d, team, teams, classes;
  float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename IN, int VPT, int FEED>
__global__ void __launch_bounds__(lnf_threads(VPT)) layer_norm_fwd_kernel(const LnfArgs a) {
  constexpr bool RING = FEED != FEED_SCALAR;
  constexpr int D = LNF_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float4 slots[2][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  const int warps = a.team >> 5, lane = t & 31;
  float4* slot = slots[0] + team_id * warps;
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  constexpr int words = VPT * Pack<IN>::WORDS;
  const Ring ring = ring_of(ring_smem, words);
  if (RING) ring_clear(ring, words, D);
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
      for (int v = 0; v < VPT; ++v)
        ring_copy<IN, FEED>(ring, stage, w, a.X, row, Cols<FEED>(v, t, a.team, d, shift), d, left);
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(row0 + i * step, i);
  }
  // FEED_SHIFT: w and b beside the ring
  IN* sw = reinterpret_cast<IN*>(ring_smem + D * ring.stage);
  const int groups = VPT * a.team;
  if (FEED == FEED_SHIFT) {
    lay_shifted<IN>(sw, 0, a.w, groups, d, shift);
    if (a.b) lay_shifted<IN>(sw, 1, a.b, groups, d, shift);
    __syncthreads();
  }
  auto vector = [&](int which, const void* from, int v, const Cols<FEED>& c) {
    if constexpr (FEED == FEED_SHIFT) return read_shifted<IN>(sw, which, groups, v * a.team + t);
    else return load8<IN, FEED>(from, 0, c, d);
  };
  // columns of this thread's warp
  float own = 0.f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
    for (int j = 0; j < 8; ++j) own += c[j] >= 0 && c[j] < d ? 1.f : 0.f;
  }
  const float cols = warp_sum(own), inv_cols = cols > 0.f ? 1.f / cols : 0.f;
  int which = 0, stage = 0;
  for (long long row = row0; row < a.T; row += step) {
    if (RING) {
      fetch(row + (D - 1) * step, stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<IN>(a.X, row + step, d, t, a.team);
    }
    float2 x[VPT][4];
    float2 s = both(0.f);
    int word = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> p = RING ? ring_read<IN, FEED>(ring, stage, word, c, d) : load8<IN, FEED>(a.X, row, c, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[v][j] = two(p, j);
        s = add2(s, x[v][j]);
      }
    }
    float mean = warp_sum(s.x + s.y) * inv_cols;
    float sq = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      if (FEED == FEED_RING) {  // a group is of the row as a whole or not at all
        float2 q = both(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = add2(x[v][j], both(-mean));
          q = fma2(y, y, q);
        }
        if (c.first < d) sq += q.x + q.y;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = (j & 1 ? x[v][j / 2].y : x[v][j / 2].x) - mean;
          if (c[j] >= 0 && c[j] < d) sq = fmaf(y, y, sq);
        }
      }
    }
    sq = warp_sum(sq);
    if (warps > 1) {
      float4* at = slot + which * 32;
      if (lane == 0) at[t >> 5] = make_float4(mean, sq, cols, 0.f);
      team_sync(team_id, a.team);
      which ^= 1;
      const float4 p = lane < warps ? at[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      mean = warp_sum(p.x * p.z) * inv_d;
      const float off = p.x - mean;
      sq = warp_sum(fmaf(p.z * off, off, p.y));
    }
    const float rstd = rsqrtf(fmaf(sq, inv_d, a.eps));
    const float2 shift_by = both(-mean), k = both(rstd);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> w = vector(0, a.w, v, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v][j] = mul2(mul2(add2(x[v][j], shift_by), k), two(w, j));
      if (a.b) {
        const Pack<IN> b = vector(1, a.b, v, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[v][j] = add2(x[v][j], two(b, j));
      }
      store8<IN, FEED>(a.Y, row, c, d, x[v]);
    }
    stage = stage + 1 < D ? stage + 1 : 0;
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
  if (RING) ring_wait<0>();
}

// Bytes of shared memory: the ring, and FEED_SHIFT's vectors.
template <typename IN>
int lnf_smem(const Geo& g, int feed) {
  if (feed == FEED_SCALAR) return 0;
  const int ring = LNF_DEPTH * Pack<IN>::WORDS * g.vpt * g.team * g.teams * 16;
  return ring + (feed == FEED_SHIFT ? 2 * g.vpt * g.team * 8 * static_cast<int>(sizeof(IN)) : 0);
}

template <typename IN, int VPT, int FEED>
cudaError_t lnf_one(const LayerNorm& n, const Geo& g) {
  const LnfArgs a = {n.X, n.w, n.b, n.Y, n.mean, n.rstd, n.T, static_cast<int>(n.d), g.team, g.teams, g.classes, n.eps};
  *n.rows = FEED_NAMES[FEED];
  auto kern = layer_norm_fwd_kernel<IN, VPT, FEED>;
  const int smem = lnf_smem<IN>(g, FEED);
  if (smem > 0) {
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
}
template <typename IN>
cudaError_t lnf_types(const LayerNorm& n) {
  const bool words = aligned16({n.X, n.w, n.b, n.Y});
  const bool shift = words && n.d % 8 != 0;
  const int64_t width = width_of(n.d, shift);
  const int vpt = width > 8192 ? LNF_MANY : groups_a_thread(n.T, width, n.num_sms, LNF_MANY);
  Geo g = geometry(n.T, n.d, shift, n.num_sms, vpt, LNF_CTA, lnf_threads(vpt));
  if (shift && lnf_smem<IN>(g, FEED_SHIFT) <= SMEM_BYTES)
    return vpt == 1 ? lnf_one<IN, 1, FEED_SHIFT>(n, g) : lnf_one<IN, LNF_MANY, FEED_SHIFT>(n, g);
  g = geometry(n.T, n.d, false, n.num_sms, vpt, LNF_CTA, lnf_threads(vpt));
  // 16,384 FP32 columns, the most there are, take 198 KB of ring
  if (!words || shift) return vpt == 1 ? lnf_one<IN, 1, FEED_SCALAR>(n, g) : lnf_one<IN, LNF_MANY, FEED_SCALAR>(n, g);
  return vpt == 1 ? lnf_one<IN, 1, FEED_RING>(n, g) : lnf_one<IN, LNF_MANY, FEED_RING>(n, g);
}

}  // namespace

cudaError_t layer_norm_fwd_launch(const LayerNorm& n) {
  switch (n.in_kind) {
    case EK_BF16: return lnf_types<__nv_bfloat16>(n);
    case EK_F16: return lnf_types<__half>(n);
    default: return lnf_types<float>(n);
  }
}

}  // namespace tg
