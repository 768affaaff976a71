// grad_clip.cu -- the norm of many gradient tensors taken as one vector, and
// their scaling to a largest norm.
//
//   norm = sqrt(sum over all elements of g^2),  c = min(1, max_norm / (norm + 1e-6))
//   out  = round(c g)
//
// Two passes over the gradients (the second needs the whole first): bound by
// HBM, with as much of the second pass as L2 still holds taken from there --
// it walks the data backwards, last read first.  1.3 GB of gradients (eight
// 2B-class layers) take 588 us out of place, 6.6 TB/s over the two reads and the
// write (chunks of 32 KB: 661 us).  The tensors are cut into
// chunks of 64 KB dealt round-robin to the CTAs, so a call costs two launches
// whatever the number of tensors (a launch takes up to 512 of them; their
// addresses travel as kernel parameters, so nothing is copied and a captured
// call needs no memory to outlive it).
//
// Sums: each thread adds squares in FP32 in two groups of 32 or 16, these in FP64; FP64
// partials of the CTAs are added in order by every CTA of the second pass, so
// results are reproducible.  A group of squares outside [2^-90, 2^120] (or
// with a value that is not finite) is added again in FP64, so neither
// overflow nor underflow of a square loses it.
#include <math.h>

#include "grad_clip.h"
#include "ptx.cuh"

namespace tg {
namespace {

constexpr int GC_THREADS = 512;
constexpr int GC_CHUNK = 65536;  // bytes
constexpr int GC_CTAS_PER_SM = 4;
constexpr int GC_FEW = 64, GC_MANY = 512;  // tensors of a launch

template <int N>
struct GradTable {
  const void* p[N];
  void* o[N];
  long long n[N];
  int cum[N + 1];  // chunks before tensor i
  unsigned char kind[N];
  int count;
};

struct Range {
  int tensor;
  long long chunk;  // of the tensor
};

template <int N>
__device__ __forceinline__ Range find_chunk(const GradTable<N>& t, int c) {
  int lo = 0, hi = t.count - 1;  // the last tensor whose chunks start at or before c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.cum[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return {lo, c - t.cum[lo]};
}

template <typename T>
__device__ __forceinline__ float gc_f(T v);
template <>
__device__ __forceinline__ float gc_f(float v) { return v; }
template <>
__device__ __forceinline__ float gc_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float gc_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void gc_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void gc_put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void gc_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Elements before the first 16-byte boundary (at most n).
template <typename T>
__device__ __forceinline__ long long head_of(const void* p, long long n) {
  const long long h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  return h < n ? h : n;
}

template <typename T>
__device__ __forceinline__ double square_d(T v) {
  const double x = static_cast<double>(gc_f(v));
  return x * x;
}

// The squares of one chunk: 16-byte words [chunk * 4096, ..) after the head;
// the first chunk also takes the head and the tail.
template <typename T>
__device__ __forceinline__ double chunk_squares(const void* base, long long n, long long chunk) {
  constexpr int V = 16 / sizeof(T);
  constexpr int WORDS = GC_CHUNK / 16;
  constexpr int PER = WORDS / GC_THREADS;  // words of a thread
  const long long head = head_of<T>(base, n);
  const long long words = (n - head) / V;
  const uint4* w = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + head);
  const long long first = chunk * WORDS + threadIdx.x;
  uint4 x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    x[i] = first + i * GC_THREADS < words ? w[first + i * GC_THREADS] : make_uint4(0, 0, 0, 0);
  float sum[2] = {0.f, 0.f};  // of 32 (FP32 elements: 16) squares each
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    any |= x[i].x | x[i].y | x[i].z | x[i].w;
    const T* e = reinterpret_cast<const T*>(&x[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) sum[i & 1] = fmaf(gc_f(e[j]), gc_f(e[j]), sum[i & 1]);
  }
  const float s = sum[0] + sum[1];  // for the range test alone: each group goes into FP64 by itself
  double d = static_cast<double>(sum[0]) + static_cast<double>(sum[1]);
  if (!(s >= 0x1p-90f && s <= 0x1p120f) && any != 0) {
    d = 0.0;
#pragma unroll 1
    for (int i = 0; i < PER; ++i) {
      const long long k = first + i * GC_THREADS;
      if (k >= words) break;
      const T* e = reinterpret_cast<const T*>(w + k);
#pragma unroll 1
      for (int j = 0; j < V; ++j) d += square_d(e[j]);
    }
  }
  if (chunk == 0) {
    const T* p = static_cast<const T*>(base);
    const long long tail = head + words * V;  // first element of the tail
    if (threadIdx.x < head) d += square_d(p[threadIdx.x]);
    if (tail + threadIdx.x < n && threadIdx.x < V) d += square_d(p[tail + threadIdx.x]);
  }
  return d;
}

// The CTA's sum, in thread 0.  FP64 adds take 16 cycles a warp here, so one
// warp adds the threads' values column by column (all warps reducing their own
// cost 10 us of a call on small tensors, with the square root in every thread).
__device__ __forceinline__ double block_sum(double d, double* s) {
  s[threadIdx.x] = d;
  __syncthreads();
  d = 0.0;
  if (threadIdx.x < 32) {
#pragma unroll
    for (int i = 0; i < GC_THREADS / 32; ++i) d += s[threadIdx.x + 32 * i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  }
  return d;
}

template <int N>
__global__ void __launch_bounds__(GC_THREADS) grad_squares_kernel(const __grid_constant__ GradTable<N> t, double* part) {
  __shared__ double s[GC_THREADS];
  pdl_wait();
  pdl_trigger();
  double d = 0.0;
  const int chunks = t.cum[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Range r = find_chunk(t, c);
    const void* p = t.p[r.tensor];
    const long long n = t.n[r.tensor];
    switch (t.kind[r.tensor]) {
      case EK_BF16: d += chunk_squares<__nv_bfloat16>(p, n, r.chunk); break;
      case EK_F16: d += chunk_squares<__half>(p, n, r.chunk); break;
      default: d += chunk_squares<float>(p, n, r.chunk); break;
    }
  }
  d = block_sum(d, s);
  if (threadIdx.x == 0) part[blockIdx.x] = d;
}

// The norm from the partials of every launch, by one warp, the same bits in every CTA.
__device__ __forceinline__ double norm_of(const double* part, int parts) {
  double d = 0.0;
  for (int i = threadIdx.x & 31; i < parts; i += 32) d += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  return sqrt(d);
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const double* part, int parts, float* norm) {
  pdl_wait();
  pdl_trigger();
  const double d = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(d);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const void* base, void* out, long long n, long long chunk, float c) {
  constexpr int V = 16 / sizeof(T);
  constexpr int WORDS = GC_CHUNK / 16;
  constexpr int PER = WORDS / GC_THREADS;
  const long long head = head_of<T>(base, n);
  const long long words = (n - head) / V;
  const T* p = static_cast<const T*>(base);
  T* o = static_cast<T*>(out);
  const long long first = chunk * WORDS + threadIdx.x;
  // the source's words are aligned; the output's only when it is off by as much
  const bool wide = ((reinterpret_cast<uintptr_t>(base) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  uint4 x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (first + i * GC_THREADS < words) x[i] = reinterpret_cast<const uint4*>(p + head)[first + i * GC_THREADS];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const long long k = first + i * GC_THREADS;
    if (k >= words) break;
    const T* e = reinterpret_cast<const T*>(&x[i]);
    if (wide) {
      uint4 y;
      T* f = reinterpret_cast<T*>(&y);
#pragma unroll
      for (int j = 0; j < V; ++j) gc_put(f + j, gc_f(e[j]) * c);
      reinterpret_cast<uint4*>(o + head)[k] = y;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) gc_put(o + head + k * V + j, gc_f(e[j]) * c);
    }
  }
  if (chunk == 0) {
    const long long tail = head + words * V;
    if (threadIdx.x < head) gc_put(o + threadIdx.x, gc_f(p[threadIdx.x]) * c);
    if (tail + threadIdx.x < n && threadIdx.x < V) gc_put(o + tail + threadIdx.x, gc_f(p[tail + threadIdx.x]) * c);
  }
}

template <int N>
__global__ void __launch_bounds__(GC_THREADS) grad_scale_kernel(const __grid_constant__ GradTable<N> t, const double* part,
                                                                int parts, float max_norm, int in_place, float* norm) {
  __shared__ float factor;
  pdl_wait();  // no early trigger: there are more CTAs than fit at once
  if (threadIdx.x < 32) {
    const double total = norm_of(part, parts);
    if (threadIdx.x == 0) {
      if (norm != nullptr && blockIdx.x == 0) *norm = static_cast<float>(total);
      const double q = static_cast<double>(max_norm) / (total + 1e-6);
      factor = static_cast<float>(q >= 1.0 ? 1.0 : q);  // not a number stays so
    }
  }
  __syncthreads();
  const float c = factor;
  if (in_place && c == 1.f) return;
  const int chunks = t.cum[t.count];
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Range r = find_chunk(t, chunks - 1 - i);
    const void* p = t.p[r.tensor];
    void* o = t.o[r.tensor];
    const long long n = t.n[r.tensor];
    switch (t.kind[r.tensor]) {
      case EK_BF16: chunk_scale<__nv_bfloat16>(p, o, n, r.chunk, c); break;
      case EK_F16: chunk_scale<__half>(p, o, n, r.chunk, c); break;
      default: chunk_scale<float>(p, o, n, r.chunk, c); break;
    }
  }
}

int64_t chunks_of(int64_t n, int kind) {
  const int64_t c = (n * elem_bytes(kind) + GC_CHUNK - 1) / GC_CHUNK;
  return c < 1 ? 1 : c;
}

// Tensors [at, at + count) of the list as one launch's table; returns how many
// fit (empty tensors are left out; *next = the first tensor not looked at).
template <int N>
int fill(const GradList& g, int64_t at, GradTable<N>* t, int64_t* next) {
  int k = 0;
  int64_t chunks = 0;
  for (; at < g.n && k < N; ++at) {
    if (g.numels[at] == 0) continue;
    const int64_t c = chunks_of(g.numels[at], g.kinds[at]);
    if (chunks + c > 0x7fffffff) break;
    t->p[k] = g.grads[at];
    t->o[k] = g.outs ? g.outs[at] : nullptr;
    t->n[k] = g.numels[at];
    t->kind[k] = static_cast<unsigned char>(g.kinds[at]);
    t->cum[k] = static_cast<int>(chunks);
    chunks += c;
    ++k;
  }
  t->cum[k] = static_cast<int>(chunks);
  t->count = k;
  *next = at;
  return k;
}

template <int N>
cudaError_t run(const GradList& g) {
  GradTable<N> t;
  const int most = GC_CTAS_PER_SM * g.num_sms;
  double* part = static_cast<double*>(g.ws);
  int parts = 0;
  for (int64_t at = 0; at < g.n;) {
    if (fill(g, at, &t, &at) == 0) continue;
    const int grid = t.cum[t.count] < most ? t.cum[t.count] : most;
    const cudaError_t e = launch_k(grad_squares_kernel<N>, dim3(grid), dim3(GC_THREADS), 0, g.stream, t, part + parts);
    if (e != cudaSuccess) return e;
    parts += grid;
  }
  bool told = false;
  if (g.outs != nullptr) {
    const bool in_place = [&] {
      for (int64_t i = 0; i < g.n; ++i)
        if (g.numels[i] > 0 && g.grads[i] != g.outs[i]) return false;
      return true;
    }();
    for (int64_t at = 0; at < g.n;) {
      if (fill(g, at, &t, &at) == 0) continue;
      const int grid = t.cum[t.count] < most ? t.cum[t.count] : most;
      const cudaError_t e = launch_k(grad_scale_kernel<N>, dim3(grid), dim3(GC_THREADS), 0, g.stream, t,
                                     static_cast<const double*>(part), parts, g.max_norm, in_place ? 1 : 0,
                                     told ? static_cast<float*>(nullptr) : g.norm);
      if (e != cudaSuccess) return e;
      told = true;
    }
  }
  if (told) return cudaSuccess;
  return launch_k(grad_norm_kernel, dim3(1), dim3(32), 0, g.stream, static_cast<const double*>(part), parts, g.norm);
}

}  // namespace

size_t grad_norm_ws_bytes(int64_t n, int num_sms) {
  // a launch takes up to GC_MANY tensors (fewer only when their chunks pass 2^31)
  const int64_t launches = (n + GC_MANY - 1) / GC_MANY + 1;
  return static_cast<size_t>(launches) * GC_CTAS_PER_SM * num_sms * sizeof(double);
}

cudaError_t grad_clip_launch(const GradList& g) { return g.n <= GC_FEW ? run<GC_FEW>(g) : run<GC_MANY>(g); }

}  // namespace tg
