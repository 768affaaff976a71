// layer_norm_fwd.cu -- layer norm over the rows of X:
//   mean = sum_c X / d,  rstd = (sum_c (X - mean)^2 / d + eps)^-1/2
//   Y    = (X - mean) rstd w + b
// FP32 arithmetic, every output rounded once.  The squares are taken of
// distances from a mean, never of X itself, so a row far from zero keeps its
// variance; a row still costs one exchange between its warps: each warp takes
// its own columns' mean and the squares around that, and the warps' pairs (of
// n_w columns, mean m_w, squares M_w) join as
//   mean = sum n_w m_w / d,   M = sum (M_w + n_w (m_w - mean)^2).
// Bound by HBM: a value read and a value written an element.  Measured: 65,536 x 2,304
// bf16 97 us, 6.2 TB/s; 16,384 x 2,304 29.8 us (a copy 23.8), 5.1 TB/s: 7 us of a call are
// its first loads and last stores; 8,192 x 2,304 FP32 30.9 us; 16,384 x 576 12.2 us; rows off
// 16 bytes 16,384 x 2,301 54 us; 8 x 576 2.1 us.
#include "layer_norm.h"
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

constexpr int LNF_MANY = 3;   // groups of eight columns a thread where rows are many or wide
constexpr int lnf_threads(int vpt, int rows) { return vpt == 1 ? 1024 : rows == 2 ? 512 : 768; }
// A CTA of several rows; with two rows at a time of 16-bit values one large CTA an SM
// (16,384 x 2,304 29.8 us, with 384 threads 32.6; FP32 8,192 x 2,304 32.3 and 30.9).
constexpr int lnf_cta(int rows, int bytes) { return rows == 2 && bytes == 2 ? 512 : 384; }
constexpr int LNF_DEPTH = 2;  // stages of the ring

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

// ROWS rows of a team at a time: their sums are exchanged together, and w and b are
// taken once for all of them.
template <typename IN, int VPT, int FEED, int ROWS>
__global__ void __launch_bounds__(lnf_threads(VPT, ROWS)) layer_norm_fwd_kernel(const LnfArgs a) {
  constexpr bool RING = FEED != FEED_SCALAR;
  constexpr int D = LNF_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float4 slots[2][32];  // of each warp: mean and squares of two rows
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  const int warps = a.team >> 5, lane = t & 31;
  float4* slot = slots[0] + team_id * warps;
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  constexpr int words = ROWS * VPT * Pack<IN>::WORDS;
  const Ring ring = ring_of(ring_smem, words);
  if (RING) ring_clear(ring, words, D);
  pdl_wait();
  pdl_trigger();
  // rows: those congruent to `cls` modulo a.classes, dealt to the teams of the CTAs with that class in turn
  const int cls = blockIdx.x % a.classes;
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  const long long row0 = cls + static_cast<long long>(a.classes) * ((blockIdx.x / a.classes) * a.teams + team_id);
  const int shift = FEED == FEED_SHIFT ? static_cast<int>((static_cast<long long>(cls) * d) & 7) : 0;
  // addresses of the row to ask for and of the row at work move on by additions
  const long long stride = step * d;
  const IN* ask = static_cast<const IN*>(a.X) + row0 * d;
  long long ask_row = row0;
  auto fetch = [&](int stage) {
    int w = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r, ask_row += step, ask += stride) {
      if (ask_row < a.T) {
        int left = 1 << 30;
        if (FEED == FEED_SHIFT && (a.T - ask_row) * d < left) left = static_cast<int>((a.T - ask_row) * d);
        int at = w;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
          ring_copy<IN, FEED>(ring, stage, at, ask, 0, Cols<FEED>(v, t, a.team, d, shift), d, left);
      }
      w += VPT * Pack<IN>::WORDS;
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(i);
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
  // columns of warp `lane` of the team, and of this one (counted element by element this
  // took 5 us of every call)
  float cols_of_lane = 0.f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const Cols<FEED> c(v, lane * 32, a.team, d, shift);
    if (FEED != FEED_SCALAR || (d & 7) == 0) {  // 256 columns from c.first on
      cols_of_lane += static_cast<float>(min(max(d - c.first, 0), 256) - max(-c.first, 0));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) cols_of_lane += static_cast<float>(min(max(d - c[j], 0), 32));
    }
  }
  if (lane >= warps) cols_of_lane = 0.f;
  const float cols = __shfl_sync(~0u, cols_of_lane, t >> 5), inv_cols = cols > 0.f ? 1.f / cols : 0.f;
  int which = 0, stage = 0;
  const IN* xr = static_cast<const IN*>(a.X) + row0 * d;
  IN* yr = static_cast<IN*>(a.Y) + row0 * d;
  for (long long row = row0; row < a.T; row += ROWS * step, xr += ROWS * stride, yr += ROWS * stride) {
    if (RING) {
      fetch(stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<IN>(a.X, row + step, d, t, a.team);
    }
    float2 x[ROWS][VPT][4];
    float mean[ROWS], sq[ROWS];
    int word = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
        const Pack<IN> p = RING ? ring_read<IN, FEED>(ring, stage, word, c, d) : load8<IN, FEED>(xr, 0, c, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[r][v][j] = two(p, j);
          s = add2(s, x[r][v][j]);
        }
      }
      mean[r] = s.x + s.y;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) mean[r] = warp_sum(mean[r]) * inv_cols;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      sq[r] = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
        if (FEED == FEED_RING) {  // a group is of the row as a whole or not at all
          float2 q = both(0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = add2(x[r][v][j], both(-mean[r]));
            q = fma2(y, y, q);
          }
          if (c.first < d) sq[r] += q.x + q.y;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = (j & 1 ? x[r][v][j / 2].y : x[r][v][j / 2].x) - mean[r];
            if (c[j] >= 0 && c[j] < d) sq[r] = fmaf(y, y, sq[r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sq[r] = warp_sum(sq[r]);
    if (warps > 1) {
      float4* at = slot + which * 32;
      if (lane == 0) at[t >> 5] = make_float4(mean[0], sq[0], mean[ROWS - 1], sq[ROWS - 1]);
      team_sync(team_id, a.team);
      which ^= 1;
      const float4 p = lane < warps ? at[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) mean[r] = warp_sum((r ? p.z : p.x) * cols_of_lane) * inv_d;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float off = (r ? p.z : p.x) - mean[r];
        sq[r] = warp_sum(fmaf(cols_of_lane * off, off, r ? p.w : p.y));
      }
    }
    float rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) rstd[r] = rsqrtf(fmaf(sq[r], inv_d, a.eps));
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> w = vector(0, a.w, v, c), b = a.b ? vector(1, a.b, v, c) : zeros<IN>();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 wj = two(w, j), bj = two(b, j);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) x[r][v][j] = fma2(add2(x[r][v][j], both(-mean[r])), mul2(wj, both(rstd[r])), bj);
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (r == 0 || row + r * step < a.T) store8<IN, FEED>(yr + r * stride, 0, c, d, x[r][v]);
    }
    stage = stage + 1 < D ? stage + 1 : 0;
    if (t == 0) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (r == 0 || row + r * step < a.T) {
          if (a.mean) a.mean[row + r * step] = mean[r];
          if (a.rstd) a.rstd[row + r * step] = rstd[r];
        }
    }
  }
  if (RING) ring_wait<0>();
}

// Bytes of shared memory: the ring, and FEED_SHIFT's vectors.
template <typename IN>
int lnf_smem(const Geo& g, int feed, int rows) {
  if (feed == FEED_SCALAR) return 0;
  const int ring = LNF_DEPTH * rows * Pack<IN>::WORDS * g.vpt * g.team * g.teams * 16;
  return ring + (feed == FEED_SHIFT ? 2 * g.vpt * g.team * 8 * static_cast<int>(sizeof(IN)) : 0);
}

template <typename IN, int VPT, int FEED, int ROWS>
cudaError_t lnf_one(const LayerNorm& n, const Geo& g) {
  const LnfArgs a = {n.X, n.w, n.b, n.Y, n.mean, n.rstd, n.T, static_cast<int>(n.d), g.team, g.teams, g.classes, n.eps};
  *n.rows = FEED_NAMES[FEED];
  auto kern = layer_norm_fwd_kernel<IN, VPT, FEED, ROWS>;
  const int smem = lnf_smem<IN>(g, FEED, ROWS);
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
  Geo g;
  auto fits = [&](int feed, int rows) {
    g = geometry(n.T, n.d, feed == FEED_SHIFT, n.num_sms, vpt, lnf_cta(rows, sizeof(IN)), lnf_threads(vpt, rows));
    return g.team * g.teams <= lnf_threads(vpt, rows) && lnf_smem<IN>(g, feed, rows) <= SMEM_BYTES;
  };
  // two rows at a time where a team has several, and one thread's registers hold them
  if (words && vpt == LNF_MANY) {
    if (fits(shift ? FEED_SHIFT : FEED_RING, 2) && n.T >= 4 * static_cast<int64_t>(g.ctas) * g.teams)
      return shift ? lnf_one<IN, LNF_MANY, FEED_SHIFT, 2>(n, g) : lnf_one<IN, LNF_MANY, FEED_RING, 2>(n, g);
  }
  if (shift && fits(FEED_SHIFT, 1))
    return vpt == 1 ? lnf_one<IN, 1, FEED_SHIFT, 1>(n, g) : lnf_one<IN, LNF_MANY, FEED_SHIFT, 1>(n, g);
  // 16,384 FP32 columns, the most there are, take 132 KB of ring
  fits(FEED_RING, 1);
  if (!words || shift) return vpt == 1 ? lnf_one<IN, 1, FEED_SCALAR, 1>(n, g) : lnf_one<IN, LNF_MANY, FEED_SCALAR, 1>(n, g);
  return vpt == 1 ? lnf_one<IN, 1, FEED_RING, 1>(n, g) : lnf_one<IN, LNF_MANY, FEED_RING, 1>(n, g);
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
