// grad_clip.cu - the global norm of many tensors (mt_grad_norm) and their
// clipping (mt_grad_clip).
#include <math.h>

#include "ops8.cuh"

namespace {

#define GC_THREADS 512
#define GC_UNIT 8192              // elements: what work is dealt out in
#define GC_PARTS 512              // partial sums of one launch, at most
#define GC_TABLE 1024             // tensors of one launch, at most

// The tensors of a launch, by value: nothing is copied to the device ahead of a
// launch, and a captured one keeps its own.
template <int N>
struct Table {
  const void* in[N];
  void* out[N];
  long long numel[N];
  uint32_t start[N + 1];          // first unit of each
  uint8_t bf16[N];
  int n;
};

// Units first..last-1 of CTA b: as many for each, within one.
__device__ __forceinline__ uint32_t gc_share(uint32_t units, uint32_t b) {
  return (uint32_t)((uint64_t)units * b / gridDim.x);
}
// the tensor that unit u lies in
template <int N>
__device__ __forceinline__ int gc_find(const Table<N>& t, uint32_t u) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}
// elements up to the next boundary of eight
template <class T>
__device__ __forceinline__ int gc_head(const T* p, long long n) {
  const int h = (int)((0 - (uintptr_t)p / sizeof(T)) & 7);
  return h < n ? h : (int)n;
}
__device__ __forceinline__ float gc_f(float v) { return v; }
__device__ __forceinline__ float gc_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Squares of n elements.  Sums of 32 bits over at most 64 squares in each of
// eight places, joined in 64; eights whose largest magnitude is over 2^52 or
// under 2^-48, where squares or their sums leave the normal numbers, are squared
// in 64 bits at once (infinities and NaN among them).
template <class T>
__device__ __forceinline__ double gc_squares(const T* p, long long n) {
  double d = 0.0;
  const int head = gc_head(p, n);
  if ((int)threadIdx.x < head) {
    const double v = gc_f(p[threadIdx.x]);
    d = v * v;
  }
  const long long vecs = (n - head) / 8;
  const T* q = p + head;
  const int tail = (int)(n - head - vecs * 8);
  if ((int)threadIdx.x < tail) {
    const double v = gc_f(q[vecs * 8 + threadIdx.x]);
    d += v * v;
  }
  constexpr int U = 4;
  for (long long i0 = threadIdx.x; i0 < vecs; i0 += 16 * U * GC_THREADS) {
    float s[8] = {};
    for (int k = 0; k < 16; ++k) {
      const long long i = i0 + (long long)k * U * GC_THREADS;
      if (i >= vecs) break;
      Raw8<T> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * GC_THREADS < vecs) v[u].template load<2>(q + (i + u * GC_THREADS) * 8, 0, 8);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u * GC_THREADS >= vecs) break;
        float x[8];
        v[u].values(x);
        const uint32_t top = v[u].top();
        if (top - 0x27800000u < 0x59800000u - 0x27800000u) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = fmaf(x[e], x[e], s[e]);
        } else if (top) {
          for (int e = 0; e < 8; ++e) d += (double)x[e] * (double)x[e];
        }
      }
    }
    d += (((double)s[0] + s[1]) + ((double)s[2] + s[3])) + (((double)s[4] + s[5]) + ((double)s[6] + s[7]));
  }
  return d;
}

// sum over the CTA, in a fixed order; every thread gets it
__device__ __forceinline__ double gc_cta_sum(double d) {
  __shared__ double red[GC_THREADS / 32];
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
  for (int i = 0; i < GC_THREADS / 32; ++i) d += red[i];
  return d;
}

template <int N>
__global__ void __launch_bounds__(GC_THREADS, 2) squares_k(const __grid_constant__ Table<N> t, double* parts) {
  ops_begin();
  const uint32_t units = t.start[t.n];
  uint32_t u = gc_share(units, blockIdx.x);
  const uint32_t end = gc_share(units, blockIdx.x + 1);
  double d = 0.0;
  if (u < end) {
    for (int s = gc_find(t, u); u < end; ++s) {
      const uint32_t first = t.start[s], last = t.start[s + 1] < end ? t.start[s + 1] : end;
      if (last <= u) continue;
      const long long lo = (long long)(u - first) * GC_UNIT, to = (long long)(last - first) * GC_UNIT;
      const long long n = (to < t.numel[s] ? to : t.numel[s]) - lo;
      d += t.bf16[s] ? gc_squares((const __nv_bfloat16*)t.in[s] + lo, n) : gc_squares((const float*)t.in[s] + lo, n);
      u = last;
    }
  }
  d = gc_cta_sum(d);
  if (threadIdx.x == 0) parts[blockIdx.x] = d;
}

struct Clip {
  const double* parts;
  float* stats;
  double scale, max_norm, eps;
  int n_parts, clip;
};
// the norm from the parts, in their order, and the factor of the clipped tensors
__device__ __forceinline__ float gc_factor(const Clip& c, bool write) {
  double d = 0.0;
  for (int i = threadIdx.x; i < c.n_parts; i += GC_THREADS) d += c.parts[i];
  const double norm = fabs(c.scale) * sqrt(gc_cta_sum(d));
  const double r = c.max_norm / (norm + c.eps), coef = r >= 1.0 ? 1.0 : r;          // NaN stays
  if (write && threadIdx.x == 0) {
    c.stats[0] = (float)norm;
    if (c.clip) c.stats[1] = (float)coef;
  }
  return (float)(c.scale * coef);
}
__global__ void __launch_bounds__(GC_THREADS) norm_k(Clip c) {
  ops_begin();
  gc_factor(c, true);
}

template <class T>
__device__ __forceinline__ T gc_t(float v);
template <>
__device__ __forceinline__ float gc_t<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 gc_t<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T>
__device__ __forceinline__ void gc_scale(const T* p, T* o, long long n, float f) {
  const int head = gc_head(p, n);
  if (head != gc_head(o, n)) {            // the two never reach a boundary together
    for (long long i = threadIdx.x; i < n; i += GC_THREADS) o[i] = gc_t<T>(gc_f(p[i]) * f);
    return;
  }
  if ((int)threadIdx.x < head) o[threadIdx.x] = gc_t<T>(gc_f(p[threadIdx.x]) * f);
  const long long vecs = (n - head) / 8;
  const int tail = (int)(n - head - vecs * 8);
  p += head;
  o += head;
  if ((int)threadIdx.x < tail) o[vecs * 8 + threadIdx.x] = gc_t<T>(gc_f(p[vecs * 8 + threadIdx.x]) * f);
  constexpr int U = 4;
  for (long long i = threadIdx.x; i < vecs; i += U * GC_THREADS) {
    Raw8<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * GC_THREADS < vecs) v[u].template load<2>(p + (i + u * GC_THREADS) * 8, 0, 8);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * GC_THREADS >= vecs) break;
      float x[8];
      v[u].values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f;
      ops_st8<2>(o + (i + u * GC_THREADS) * 8, 0, 8, x);
    }
  }
}

template <int N>
__global__ void __launch_bounds__(GC_THREADS, 2) scale_k(const __grid_constant__ Table<N> t, Clip c, int first) {
  ops_begin();
  const float f = gc_factor(c, first && blockIdx.x == 0);
  const uint32_t units = t.start[t.n];
  uint32_t u = gc_share(units, blockIdx.x);
  const uint32_t end = gc_share(units, blockIdx.x + 1);
  if (u >= end) return;
  for (int s = gc_find(t, u); u < end; ++s) {
    const uint32_t from = t.start[s], last = t.start[s + 1] < end ? t.start[s + 1] : end;
    if (last <= u) continue;
    const long long lo = (long long)(u - from) * GC_UNIT, to = (long long)(last - from) * GC_UNIT;
    const long long n = (to < t.numel[s] ? to : t.numel[s]) - lo;
    u = last;
    if (f == 1.f && t.in[s] == t.out[s]) continue;          // in place and nothing to clip
    if (t.bf16[s]) gc_scale((const __nv_bfloat16*)t.in[s] + lo, (__nv_bfloat16*)t.out[s] + lo, n, f);
    else gc_scale((const float*)t.in[s] + lo, (float*)t.out[s] + lo, n, f);
  }
}

int spans_ok(const mt_span* s, int32_t n, bool out) {
  if (n < 0 || (n && !s)) return MT_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    if (s[i].numel < 0 || !ops_dtype_ok(s[i].dtype) || s[i].reserved0) return MT_ERR_ARG;
    if (s[i].numel > (1LL << 40)) return MT_ERR_UNSUPPORTED;
    const int es = ops_size(s[i].dtype);
    if (s[i].numel && (!s[i].grad || !ops_aligned(s[i].grad, es))) return MT_ERR_ARG;
    if (s[i].numel && out && (!s[i].out || !ops_aligned(s[i].out, es))) return MT_ERR_ARG;
  }
  return MT_OK;
}
template <int N>
void fill(Table<N>& t, const mt_span* s, int n) {
  uint32_t u = 0;
  for (int i = 0; i < n; ++i) {
    t.in[i] = s[i].grad;
    t.out[i] = s[i].out;
    t.numel[i] = s[i].numel;
    t.bf16[i] = s[i].dtype == MT_DT_BF16;
    t.start[i] = u;
    u += (uint32_t)((s[i].numel + GC_UNIT - 1) / GC_UNIT);
  }
  t.start[n] = u;
  t.n = n;
}
unsigned gc_grid(uint32_t units, int sms) {
  const uint32_t most = (uint32_t)ops_least(2 * sms, GC_PARTS);
  return units < 1 ? 1 : units < most ? units : most;
}
// one launch over up to N tensors: squares into parts, or scaled into out
template <int N>
int launch(const mt_span* s, int n, int sms, double* parts, const Clip* c, int first, int* used, cudaStream_t st) {
  Table<N> t;
  fill(t, s, n);
  const unsigned grid = gc_grid(t.start[n], sms);
  *used = (int)grid;
  if (!c) return ops_launch(squares_k<N>, grid, GC_THREADS, 0, st, 1, t, parts);
  return ops_launch(scale_k<N>, grid, GC_THREADS, 0, st, 1, t, *c, first);
}
int launch_any(const mt_span* s, int n, int sms, double* parts, const Clip* c, int first, int* used, cudaStream_t st) {
  auto f = n <= 32 ? launch<32> : n <= 256 ? launch<256> : launch<GC_TABLE>;
  return f(s, n, sms, parts, c, first, used, st);
}
int all(const mt_span* s, int32_t n, const Clip& c0, void* ws, int64_t ws_bytes, void* stream) {
  Clip c = c0;
  if (!ws || !ops_aligned(ws, 16)) return MT_ERR_ARG;
  if (ws_bytes < mt_grad_ws_bytes(n)) return MT_ERR_ARENA_SMALL;
  // more units than 32 bits count are refused (2^45 elements)
  int64_t units = 0;
  for (int i = 0; i < n; ++i) units += (s[i].numel + GC_UNIT - 1) / GC_UNIT;
  if (units >= (1LL << 31)) return MT_ERR_UNSUPPORTED;
  int dev, sms;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_CUDA;
  }
  cudaStream_t st = (cudaStream_t)stream;
  c.parts = (const double*)ws;
  c.n_parts = 0;
  for (int i = 0; i < n; i += GC_TABLE) {
    int used = 0;
    const int rc = launch_any(s + i, ops_least(n - i, GC_TABLE), sms, (double*)ws + c.n_parts, nullptr, 0, &used, st);
    if (rc) return rc;
    c.n_parts += used;
  }
  if (!c.clip || n == 0) return ops_launch(norm_k, 1, GC_THREADS, 0, st, 1, c);
  for (int i = 0; i < n; i += GC_TABLE) {
    int used = 0;
    const int rc = launch_any(s + i, ops_least(n - i, GC_TABLE), sms, nullptr, &c, i == 0, &used, st);
    if (rc) return rc;
  }
  return MT_OK;
}

}  // namespace

extern "C" {

int64_t mt_grad_ws_bytes(int32_t n) {
  if (n < 0) return -MT_ERR_ARG;
  return ((int64_t)n + GC_TABLE) / GC_TABLE * GC_PARTS * 8;
}

int32_t mt_grad_norm(const mt_span* spans, int32_t n, double scale, float* norm, void* ws, int64_t ws_bytes,
                     void* stream) {
  const int st = spans_ok(spans, n, false);
  if (st) return st;
  if (!isfinite(scale) || !norm || !ops_aligned(norm, 4)) return MT_ERR_ARG;
  const Clip c = {nullptr, norm, scale, 1.0, 0.0, 0, 0};
  return all(spans, n, c, ws, ws_bytes, stream);
}

int32_t mt_grad_clip(const mt_span* spans, int32_t n, double max_norm, double eps, double scale, float* stats, void* ws,
                     int64_t ws_bytes, void* stream) {
  const int st = spans_ok(spans, n, true);
  if (st) return st;
  if (!(max_norm > 0) || !isfinite(max_norm) || !(eps >= 0) || !isfinite(eps) || !isfinite(scale)) return MT_ERR_ARG;
  if (!stats || !ops_aligned(stats, 4)) return MT_ERR_ARG;
  const Clip c = {nullptr, stats, scale, max_norm, eps, 0, 1};
  return all(spans, n, c, ws, ws_bytes, stream);
}

}  // extern "C"
