// norm_fwd.cu -- the norm after a block, its gate, the residual sum and the
// norm before the next block, in one pass over the rows.
//
//   u  = B rstd_b w_post             rstd_b = (mean_c B^2 + eps)^-1/2
//   H' = res_scale H + gate u
//   N  = H' rstd_h w_pre             rstd_h = (mean_c H'^2 + eps)^-1/2
// FP32 arithmetic, every output rounded once; N is taken from the unrounded
// H'.  Bound by HBM: 2 values (3 with an element-wise gate) read and 2 written
// an element.  Measured: 16,384 x 2,304 bf16 with an element-wise gate 66 us, 5.7
// TB/s; 4,096 x 5,760 37 us, 5.2 TB/s; 16,384 x 576 19 us, 4.0 TB/s; 8,192 x 2,304
// without a gate 31 us, 8,192 x 2,300 47 us; 8 x 576 2.2 us.
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

// Groups a thread: 1 (up to 8,192 columns) or 3.  Threads of a CTA, and of an
// SM (64 or 80 registers each).
constexpr int FWD_MANY = 3;
constexpr int fwd_threads(int vpt) { return vpt == 1 ? 1024 : 768; }
constexpr int FWD_CTA = 384;  // a CTA of several rows
constexpr int FWD_DEPTH = 2;  // rows in the ring

template <typename IN, typename RES, int VPT, int FEED>
__global__ void __launch_bounds__(fwd_threads(VPT)) norm_fwd_kernel(const Args a) {
  constexpr bool RING = FEED == FEED_RING || FEED == FEED_SHIFT;
  constexpr int D = FWD_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float slots[2][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  float* slot = slots[0] + team_id * (a.team >> 5);
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool full = a.gate_kind == GATE_FULL, channel = a.gate_kind == GATE_CHANNEL;
  const int ring_words = VPT * (Pack<RES>::WORDS + (full ? 2 : 1) * Pack<IN>::WORDS);
  const Ring ring = ring_of(ring_smem, ring_words);
  if (RING) ring_clear(ring, ring_words, D);
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
        ring_copy<IN, FEED>(ring, stage, w, a.B, row, c, d, left);
        ring_copy<RES, FEED>(ring, stage, w, a.H, row, c, d, left);
        if (full) ring_copy<IN, FEED>(ring, stage, w, a.gate, row, c, d, left);
      }
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(row0 + i * step, i);
  }
  // FEED_SHIFT: w_post, w_pre and a channel gate, beside the ring
  IN* sw = reinterpret_cast<IN*>(ring_smem + D * ring.stage);
  const int groups = VPT * a.team;
  if (FEED == FEED_SHIFT) {
    lay_shifted<IN>(sw, 0, a.w_post, groups, d, shift);
    lay_shifted<IN>(sw, 1, a.w_pre, groups, d, shift);
    if (channel) lay_shifted<IN>(sw, 2, a.gate, groups, d, shift);
    __syncthreads();
  }
  auto vector = [&](int which, const void* from, int v, const Cols<FEED>& c) {
    if constexpr (FEED == FEED_SHIFT) return read_shifted<IN>(sw, which, groups, v * a.team + t);
    else return load8<IN, FEED>(from, 0, c, d);
  };
  int which = 0, stage = 0;
  const bool token = a.gate_kind == GATE_TOKEN;
  float gt_next = token && row0 < a.T ? to_f(static_cast<const IN*>(a.gate)[row0]) : 1.f;
  for (long long row = row0; row < a.T; row += step) {
    const float gt = gt_next;  // loaded a row ahead
    if (token && row + step < a.T) gt_next = to_f(static_cast<const IN*>(a.gate)[row + step]);
    if (RING) {
      fetch(row + (D - 1) * step, stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<IN>(a.B, row + step, d, t, a.team);
      prefetch_row<RES>(a.H, row + step, d, t, a.team);
      if (full) prefetch_row<IN>(a.gate, row + step, d, t, a.team);
    }
    // word w of the ring's group v
    const int words = Pack<RES>::WORDS + (full ? 2 : 1) * Pack<IN>::WORDS;
    float2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      int w = v * words;
      const Pack<IN> b = RING ? ring_read<IN, FEED>(ring, stage, w, c, d) : load8<IN, FEED>(a.B, row, c, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = two(b, j);
        s = fma2(x, x, s);
      }
    }
    const float rb = rsqrtf(team_sum(s.x + s.y, slot, which, team_id, a.team, t) * inv_d + a.eps);
    which ^= 1;
    const float2 k = both(rb * gt), sc = both(a.res_scale);
    float2 x[VPT][4];
    s = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      int w = v * words;
      Pack<IN> b, g;
      Pack<RES> h;
      if (RING) {
        b = ring_read<IN, FEED>(ring, stage, w, c, d);
        h = ring_read<RES, FEED>(ring, stage, w, c, d);
        if (full) g = ring_read<IN, FEED>(ring, stage, w, c, d);
      } else {
        b = load8<IN, FEED>(a.B, row, c, d);
        h = load8<RES, FEED>(a.H, row, c, d);
        if (full) g = load8<IN, FEED>(a.gate, row, c, d);
      }
      if (channel) g = vector(2, a.gate, v, c);
      const Pack<IN> wpost = vector(0, a.w_post, v, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 u = mul2(mul2(two(b, j), k), two(wpost, j));
        if (full || channel) u = mul2(u, two(g, j));
        x[v][j] = fma2(sc, two(h, j), u);
        s = fma2(x[v][j], x[v][j], s);
      }
      store8<RES, FEED>(a.H_out, row, c, d, x[v]);
    }
    const float rh = rsqrtf(team_sum(s.x + s.y, slot, which, team_id, a.team, t) * inv_d + a.eps);
    which ^= 1;
    const float2 rh2 = both(rh);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      const Pack<IN> wpre = vector(1, a.w_pre, v, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v][j] = mul2(x[v][j], mul2(rh2, two(wpre, j)));
      store8<IN, FEED>(a.N, row, c, d, x[v]);
    }
    stage = stage + 1 < D ? stage + 1 : 0;
    if (t == 0) {
      if (a.rstd_b) a.rstd_b[row] = rb;
      if (a.rstd_h) a.rstd_h[row] = rh;
    }
  }
  if (RING) ring_wait<0>();
}

template <typename IN, typename RES>
int fwd_words(const NormResidual& n) { return Pack<RES>::WORDS + (n.gate_kind == GATE_FULL ? 2 : 1) * Pack<IN>::WORDS; }
// Bytes of shared memory: the ring, and FEED_SHIFT's vectors.
template <typename IN, typename RES>
int fwd_smem(const NormResidual& n, const Geo& g, int feed) {
  if (feed != FEED_RING && feed != FEED_SHIFT) return 0;
  const int ring = FWD_DEPTH * fwd_words<IN, RES>(n) * g.vpt * g.team * g.teams * 16;
  return ring + (feed == FEED_SHIFT ? 3 * g.vpt * g.team * 8 * static_cast<int>(sizeof(IN)) : 0);
}

template <typename IN, typename RES, int VPT, int FEED>
cudaError_t fwd_one(const NormResidual& n, const Geo& g) {
  const Args a = to_args(n, g);
  *n.rows = FEED_NAMES[FEED];
  auto kern = norm_fwd_kernel<IN, RES, VPT, FEED>;
  const int smem = fwd_smem<IN, RES>(n, g, FEED);
  if (smem > 0) {
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
}
template <typename IN, typename RES>
cudaError_t fwd_types(const NormResidual& n) {
  // a gate of one value a row needs no alignment
  const bool wide_gate = n.gate_kind == GATE_FULL || n.gate_kind == GATE_CHANNEL;
  const bool words = aligned16({n.B, n.H, n.w_post, n.w_pre, n.H_out, n.N, wide_gate ? n.gate : nullptr});
  const bool shift = words && n.d % 8 != 0;
  const int64_t width = width_of(n.d, shift);
  const int vpt = width > 8192 ? FWD_MANY : groups_a_thread(n.T, width, n.num_sms, FWD_MANY);
  Geo g = geometry(n.T, n.d, shift, n.num_sms, vpt, FWD_CTA, fwd_threads(vpt));
  if (shift && fwd_smem<IN, RES>(n, g, FEED_SHIFT) <= SMEM_BYTES)
    return vpt == 1 ? fwd_one<IN, RES, 1, FEED_SHIFT>(n, g) : fwd_one<IN, RES, FWD_MANY, FEED_SHIFT>(n, g);
  g = geometry(n.T, n.d, false, n.num_sms, vpt, FWD_CTA, fwd_threads(vpt));
  if (!words || shift) return vpt == 1 ? fwd_one<IN, RES, 1, FEED_SCALAR>(n, g) : fwd_one<IN, RES, FWD_MANY, FEED_SCALAR>(n, g);
  if (vpt == 1) return fwd_one<IN, RES, 1, FEED_RING>(n, g);  // 196 KB at most
  return fwd_smem<IN, RES>(n, g, FEED_RING) <= SMEM_BYTES ? fwd_one<IN, RES, FWD_MANY, FEED_RING>(n, g)
                                                          : fwd_one<IN, RES, FWD_MANY, FEED_VEC>(n, g);
}

}  // namespace

cudaError_t norm_residual_fwd_launch(const NormResidual& n) {
  const bool r32 = n.res_kind == EK_F32;
  switch (n.in_kind) {
    case EK_BF16: return r32 ? fwd_types<__nv_bfloat16, float>(n) : fwd_types<__nv_bfloat16, __nv_bfloat16>(n);
    case EK_F16: return r32 ? fwd_types<__half, float>(n) : fwd_types<__half, __half>(n);
    default: return fwd_types<float, float>(n);
  }
}

}  // namespace tg
