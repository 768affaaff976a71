// norm_bwd.cu -- backward of norm_fwd.cu, for dH' and dN (means over the row):
//   hn = H' rstd_h, g1 = dN w_pre,  dh = dH' + rstd_h (g1 - hn mean(g1 hn))
//   bn = B rstd_b,  du = gate dh,   g2 = du w_post
//   dB = rstd_b (g2 - bn mean(g2 bn)),  dH = res_scale dh
//   dw_pre = sum_t dN hn,  dw_post = sum_t du bn,  dgate = dh bn w_post summed
//   over what the gate was broadcast along
// FP32 arithmetic, every output rounded once; the stored H' is what the
// derivative is taken at.  Bound by HBM: 4 values (5 with an element-wise
// gate) read and 2 (3) written an element, in one pass: the column sums build
// up in registers (rows of up to 4,096 columns; in shared memory beyond, where
// 16 or 32 columns a thread would spill); the teams of a CTA are added in
// shared memory, the CTAs by a second launch, all in a fixed order.
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

constexpr int BWD_THREADS = 576;  // of a CTA: one CTA an SM (few partial sums), 18 warps
constexpr int BWD_DEPTH = 2;      // rows in the ring

__device__ __forceinline__ void put_kind(void* p, long long i, float v, int kind) {
  if (kind == EK_F32) static_cast<float*>(p)[i] = v;
  else if (kind == EK_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <typename IN, typename RES, int VPT, int FEED>
__global__ void __launch_bounds__(VPT > 1 ? MAX_TEAM : BWD_THREADS, 1) norm_bwd_kernel(const Args a) {
  constexpr bool VEC = FEED != FEED_SCALAR;
  constexpr int D = BWD_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];  // the ring, then the column sums [3][d]
  __shared__ float2 slots[MAX_TEAMS][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  float2* slot = slots[team_id];
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool full = a.gate_kind == GATE_FULL, channel = a.gate_kind == GATE_CHANNEL;
  const bool per_element = full || channel;
  const Ring ring = ring_of(ring_smem, VPT * (2 * Pack<RES>::WORDS + (full ? 3 : 2) * Pack<IN>::WORDS));
  pdl_wait();
  pdl_trigger();
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  const long long row0 = static_cast<long long>(blockIdx.x) * a.teams + team_id;
  auto fetch = [&](long long row, int stage) {
    if (row < a.T) {
      int w = 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * a.team + t) * 8;
        ring_copy<RES>(ring, stage, w, a.H, row, c, d);
        ring_copy<IN>(ring, stage, w, a.dN, row, c, d);
        ring_copy<RES>(ring, stage, w, a.dH_out, row, c, d);
        ring_copy<IN>(ring, stage, w, a.B, row, c, d);
        if (full) ring_copy<IN>(ring, stage, w, a.gate, row, c, d);
      }
    }
    ring_commit();
  };
  if (FEED == FEED_RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(row0 + i * step, i);
  }
  // VPT > 1 (one team a CTA): sum k of the thread's group v, half i at (((k * VPT + v) * 2 + i) * team + t)
  constexpr bool IN_SMEM = VPT > 1;
  const int ring_bytes = FEED == FEED_RING ? D * static_cast<int>(ring.stage) : 0;
  float4* accs = reinterpret_cast<float4*>(ring_smem + ring_bytes) + t;
  auto at = [&](int k, int v, int i) -> float4& { return accs[((k * VPT + v) * 2 + i) * a.team]; };
  auto add8 = [&](int k, int v, const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 f = at(k, v, i);
      f.x += x[4 * i];
      f.y += x[4 * i + 1];
      f.z += x[4 * i + 2];
      f.w += x[4 * i + 3];
      at(k, v, i) = f;
    }
  };
  if (IN_SMEM) {
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) at(k, v, 0) = at(k, v, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float acc_post[8] = {}, acc_pre[8] = {}, acc_gate[8] = {};
  int which = 0, stage = 0;
  for (long long row = row0; row < a.T; row += step) {
    Pack<IN> b[VPT], dn[VPT], g[VPT];
    Pack<RES> h[VPT], dho[VPT];
    const float gt = a.gate_kind == GATE_TOKEN ? to_f(static_cast<const IN*>(a.gate)[row]) : 1.f;
    const float rb = a.rstd_b[row], rh = a.rstd_h[row];
    if (FEED == FEED_RING) {
      fetch(row + (D - 1) * step, stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
      int w = 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * a.team + t) * 8;
        h[v] = ring_read<RES>(ring, stage, w, c, d);
        dn[v] = ring_read<IN>(ring, stage, w, c, d);
        dho[v] = ring_read<RES>(ring, stage, w, c, d);
        b[v] = ring_read<IN>(ring, stage, w, c, d);
        if (full) g[v] = ring_read<IN>(ring, stage, w, c, d);
      }
      stage = stage + 1 < D ? stage + 1 : 0;
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * a.team + t) * 8;
        h[v] = load8<RES, VEC>(a.H, row, c, d);
        dn[v] = load8<IN, VEC>(a.dN, row, c, d);
        dho[v] = load8<RES, VEC>(a.dH_out, row, c, d);
        b[v] = load8<IN, VEC>(a.B, row, c, d);
        if (full) g[v] = load8<IN, VEC>(a.gate, row, c, d);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      const Pack<IN> wpre = load8<IN, VEC>(a.w_pre, 0, c, d);
      if (channel) g[v] = load8<IN, VEC>(a.gate, 0, c, d);
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = to_f(dn[v].v[j]) * (to_f(h[v].v[j]) * rh);
        if (!IN_SMEM) acc_pre[j] += p[j];
        s = fmaf(p[j], to_f(wpre.v[j]), s);
      }
      if (IN_SMEM) add8(1, v, p);
    }
    s = team_sum(make_float2(s, 0.f), slot, which, team_id, a.team, t).x;
    which ^= 1;
    const float m1 = s * inv_d;
    float dh[VPT][8];
    float2 s2 = make_float2(0.f, 0.f);  // (sum of g2 bn, sum of dgate)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      const Pack<IN> wpre = load8<IN, VEC>(a.w_pre, 0, c, d);
      const Pack<IN> wpost = load8<IN, VEC>(a.w_post, 0, c, d);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hn = to_f(h[v].v[j]) * rh;
        const float x = to_f(dho[v].v[j]) + rh * (to_f(dn[v].v[j]) * to_f(wpre.v[j]) - hn * m1);
        o[j] = a.res_scale * x;
        dh[v][j] = x;
      }
      store8<RES, VEC>(a.dH, row, c, d, o);
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float bn = to_f(b[v].v[j]) * rb;
        const float e = dh[v][j] * bn;          // dw_post's term before the gate
        const float dg = e * to_f(wpost.v[j]);  // the gate's gradient, element by element
        const float gg = per_element ? to_f(g[v].v[j]) : gt;
        q[j] = gg * e;
        if (!IN_SMEM) acc_post[j] += q[j];
        s2.x = fmaf(gg, dg, s2.x);
        s2.y += dg;
        if (!IN_SMEM && channel) acc_gate[j] += dg;
        o[j] = dg;
      }
      if (IN_SMEM) {
        add8(0, v, q);
        if (channel) add8(2, v, o);
      }
      if (full) store8<IN, VEC>(a.dgate, row, c, d, o);
    }
    s2 = team_sum(s2, slot, which, team_id, a.team, t);
    which ^= 1;
    if (a.gate_kind == GATE_TOKEN && t == 0) put_kind(a.dgate, row, s2.y, a.out_kind);
    const float m2 = s2.x * inv_d;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      const Pack<IN> wpost = load8<IN, VEC>(a.w_post, 0, c, d);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gg = per_element ? to_f(g[v].v[j]) : gt;
        const float bn = to_f(b[v].v[j]) * rb;
        o[j] = rb * (gg * dh[v][j] * to_f(wpost.v[j]) - bn * m2);
      }
      store8<IN, VEC>(a.dB, row, c, d, o);
    }
  }
  if (FEED == FEED_RING) ring_wait<0>();
  const int sums = channel ? 3 : 2;
  float* out = a.part + static_cast<long long>(blockIdx.x) * 3 * d;
  if (IN_SMEM) {
    for (int k = 0; k < sums; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * a.team + t) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 f = at(k, v, i);
          float* p = out + k * d + c + 4 * i;
          if (c + 4 * i < d) p[0] = f.x;
          if (c + 4 * i + 1 < d) p[1] = f.y;
          if (c + 4 * i + 2 < d) p[2] = f.z;
          if (c + 4 * i + 3 < d) p[3] = f.w;
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
      for (int j = 0; j < 8; ++j)
        if (t * 8 + j < d) {
          float* p = col + t * 8 + j;
          p[0] = (k ? p[0] : 0.f) + acc_post[j];
          p[d] = (k ? p[d] : 0.f) + acc_pre[j];
          if (channel) p[2 * d] = (k ? p[2 * d] : 0.f) + acc_gate[j];
        }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < sums * d; i += blockDim.x) out[i] = col[i];
}

// Column sums of the CTAs' partials [ctas][3][d], a block of 32 columns per
// CTA: 8 threads a column add every eighth partial in order, then each other.
__global__ void __launch_bounds__(256) norm_cols_kernel(const float* part, int ctas, int d, int sums, void* dw_post,
                                                        void* dw_pre, void* dgate, int kind) {
  __shared__ float s[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + x;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (i < sums * d) {
#pragma unroll 4
    for (int c = y; c < ctas; c += 8) v += part[static_cast<long long>(c) * 3 * d + i];
  }
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && i < sums * d) {
    for (int k = 1; k < 8; ++k) v += s[k][x];
    const int which = i / d;
    put_kind(which == 0 ? dw_post : which == 1 ? dw_pre : dgate, i - which * d, v, kind);
  }
}

Geo bwd_geometry(int64_t T, int64_t d, int sms) {
  Geo g = geometry(T, d, sms, BWD_THREADS, 1);
  if (g.vpt > 1) {  // one row at a time
    g.teams = 1;
    g.ctas = static_cast<int>(T < sms ? T : sms);
  }
  return g;
}
// Bytes of the ring and of the column sums beside it (VPT > 1) or in its place.
int ring_bytes(const Geo& g, int words) { return BWD_DEPTH * words * g.team * g.teams * 16; }
int sum_bytes(const Geo& g, int64_t d) { return static_cast<int>(g.vpt > 1 ? 3 * g.vpt * g.team * 32 : 3 * d * 4); }

template <typename IN, typename RES, int VPT, int FEED>
cudaError_t bwd_one(const NormResidual& n, const Geo& g) {
  const Args a = to_args(n, g);
  auto kern = norm_bwd_kernel<IN, RES, VPT, FEED>;
  const int words = VPT * (2 * Pack<RES>::WORDS + (n.gate_kind == GATE_FULL ? 3 : 2) * Pack<IN>::WORDS);
  const int ring = FEED == FEED_RING ? ring_bytes(g, words) : 0, sums_at = sum_bytes(g, n.d);
  const int smem = VPT > 1 ? ring + sums_at : ring > sums_at ? ring : sums_at;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  e = launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
  if (e != cudaSuccess) return e;
  const int sums = n.gate_kind == GATE_CHANNEL ? 3 : 2;
  return launch_k(norm_cols_kernel, dim3(static_cast<unsigned>((sums * n.d + 31) / 32)), dim3(256), 0, n.stream,
                  static_cast<const float*>(n.ws), g.ctas, static_cast<int>(n.d), sums, n.dw_post, n.dw_pre, n.dgate,
                  n.out_kind);
}
template <typename IN, typename RES>
cudaError_t bwd_types(const NormResidual& n) {
  Geo g = bwd_geometry(n.T, n.d, n.num_sms);
  const bool full = n.gate_kind == GATE_FULL, wide_gate = full || n.gate_kind == GATE_CHANNEL;
  const bool vec = vec_ok({n.B, n.H, n.w_post, n.w_pre, n.dH_out, n.dN, n.dB, n.dH, wide_gate ? n.gate : nullptr,
                           full ? n.dgate : nullptr},
                          n.d);
  const int words = g.vpt * (2 * Pack<RES>::WORDS + (full ? 3 : 2) * Pack<IN>::WORDS);
  while (g.teams > 1 && ring_bytes(g, words) > SMEM_BYTES) --g.teams;  // fewer rows at once
  const bool ring = vec && ring_bytes(g, words) + (g.vpt > 1 ? sum_bytes(g, n.d) : 0) <= SMEM_BYTES;
  switch (g.vpt) {
    case 1: return ring ? bwd_one<IN, RES, 1, FEED_RING>(n, g) : bwd_one<IN, RES, 1, FEED_SCALAR>(n, g);
    case 2:
      return ring  ? bwd_one<IN, RES, 2, FEED_RING>(n, g)
             : vec ? bwd_one<IN, RES, 2, FEED_VEC>(n, g)
                   : bwd_one<IN, RES, 2, FEED_SCALAR>(n, g);
    default: return vec ? bwd_one<IN, RES, 4, FEED_VEC>(n, g) : bwd_one<IN, RES, 4, FEED_SCALAR>(n, g);
  }
}

}  // namespace

size_t norm_residual_bwd_ws_bytes(int64_t T, int64_t d, int num_sms) {
  if (T <= 0 || d <= 0) return 0;
  return static_cast<size_t>(bwd_geometry(T, d, num_sms).ctas) * 3 * d * 4;
}

cudaError_t norm_residual_bwd_launch(const NormResidual& n) {
  const bool r32 = n.res_kind == EK_F32;
  switch (n.in_kind) {
    case EK_BF16: return r32 ? bwd_types<__nv_bfloat16, float>(n) : bwd_types<__nv_bfloat16, __nv_bfloat16>(n);
    case EK_F16: return r32 ? bwd_types<__half, float>(n) : bwd_types<__half, __half>(n);
    default: return bwd_types<float, float>(n);
  }
}

}  // namespace tg
