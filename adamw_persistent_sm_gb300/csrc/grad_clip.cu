// grad_clip.cu - the global norm of many tensors (mt_grad_norm) and their
// clipping (mt_grad_clip).
#include <math.h>

#include "ops8.cuh"

namespace {

#define GC_THREADS 256
#define GC_CTAS 3                 // of an SM (219M fp32 elements: 399 us, in the same run four 408)
#define GC_UNIT 8192              // elements: what work is dealt out in
#define GC_PARTS 1024              // partial sums of one launch, at most
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

// A thread's sum of squares.  In 32 bits over at most 64 squares in each of eight
// places, then joined in 64; eights whose largest magnitude is over 2^52 or under
// 2^-48, where squares or their sums leave the normal numbers, are squared in 64 bits
// at once (infinities and NaN among them).  Sixty-four-bit instructions are some
// thirty times slower here: with eight of them for every run of a tensor and a
// reduction of all threads in 64 bits, 16 MB of 500 tensors took 34 us.
#define GC_JOIN 64
struct Squares {
  float s[8];
  double d;
  int n;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    d = 0.0;
    n = 0;
  }
  __device__ __forceinline__ float places() {
    const float t = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    n = 0;
    return t;
  }
  __device__ __forceinline__ void room(int more) {
    if (n + more > GC_JOIN) d += (double)places();
    n += more;
  }
  __device__ __forceinline__ static bool plain(uint32_t top) { return top - 0x27800000u < 0x59800000u - 0x27800000u; }
  __device__ __forceinline__ void one(float x) {
    const uint32_t top = __float_as_uint(x) & 0x7fffffffu;
    if (plain(top)) s[0] = fmaf(x, x, s[0]);
    else if (top) d += (double)x * (double)x;
  }
  template <class T>
  __device__ __forceinline__ void eight(const Raw8<T>& v) {
    float x[8];
    v.values(x);
    const uint32_t top = v.top();
    if (plain(top)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = fmaf(x[e], x[e], s[e]);
    } else if (top) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d += (double)x[e] * (double)x[e];
    }
  }
};

#define GC_FLIGHT 4               // eights of a thread on their way at once (219M fp32: 404 us, in the same
                                  // run two 425; 500 ragged bf16 tensors: 26 us, three 29)
// n elements at p
template <class T>
__device__ __forceinline__ void gc_squares(Squares& q, const T* p, long long n) {
  const int head = gc_head(p, n);
  const long long vecs = (n - head) / 8;
  const int tail = (int)(n - head - vecs * 8);
  q.room(2);
  if ((int)threadIdx.x < head) q.one(gc_f(p[threadIdx.x]));
  p += head;
  if ((int)threadIdx.x < tail) q.one(gc_f(p[vecs * 8 + threadIdx.x]));
  for (long long i = threadIdx.x; i < vecs; i += GC_FLIGHT * GC_THREADS) {
    Raw8<T> v[GC_FLIGHT];
#pragma unroll
    for (int u = 0; u < GC_FLIGHT; ++u)
      if (i + u * GC_THREADS < vecs) v[u].template load<2>(p + (i + u * GC_THREADS) * 8, 0, 8);
    q.room(GC_FLIGHT);
#pragma unroll
    for (int u = 0; u < GC_FLIGHT; ++u)
      if (i + u * GC_THREADS < vecs) q.eight(v[u]);
  }
}

// A CTA takes a contiguous run of units, over as many tensors as lie in it.  876 MB of
// fp32: 128 us, the copy rate; 438 MB of bf16, with half the bytes on their way, 75, 86 %
// of it.
template <int N>
__global__ void __launch_bounds__(GC_THREADS, GC_CTAS) squares_k(const __grid_constant__ Table<N> t, double* parts) {
  ops_begin();
  __shared__ double red[GC_THREADS / 32];
  const uint32_t units = t.start[t.n];
  uint32_t u = gc_share(units, blockIdx.x);
  const uint32_t end = gc_share(units, blockIdx.x + 1);
  Squares q;
  q.clear();
  if (u < end) {
    for (int s = gc_find(t, u); u < end; ++s) {
      const uint32_t first = t.start[s], last = t.start[s + 1] < end ? t.start[s + 1] : end;
      if (last <= u) continue;
      const long long lo = (long long)(u - first) * GC_UNIT, to = (long long)(last - first) * GC_UNIT;
      const long long n = (to < t.numel[s] ? to : t.numel[s]) - lo;
      if (t.bf16[s]) gc_squares(q, (const __nv_bfloat16*)t.in[s] + lo, n);
      else gc_squares(q, (const float*)t.in[s] + lo, n);
      u = last;
    }
  }
  // the CTA's threads, in 32 bits where no thread has more, then its warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (__syncthreads_or(q.d != 0.0)) {
    double d = q.d + (double)q.places();
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) red[warp] = d;
  } else {
    float f = q.places();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    if (lane == 0) red[warp] = (double)f;
  }
  __syncthreads();
  if (warp) return;
  double d = lane < GC_THREADS / 32 ? red[lane] : 0.0;
  for (int o = GC_THREADS / 64; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) parts[blockIdx.x] = d;
}

struct Clip {
  const double* parts;
  float* stats;
  double scale, max_norm, eps;
  int n_parts, clip;
};
// The norm from the parts, in their order, and the factor of the clipped tensors: by
// one warp, for the CTA.  In 32 bits where they hold the sum, its root, the limit and eps.
__device__ __forceinline__ float gc_factor(const Clip& c, bool write) {
  __shared__ float factor;
  if (threadIdx.x < 32) {
    double d = 0.0;
    for (int i0 = 0; i0 < c.n_parts; i0 += 512) {
      double v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = i0 + u * 32 + (int)threadIdx.x < c.n_parts ? __ldcg(c.parts + i0 + u * 32 + threadIdx.x) : 0.0;
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (i0 + u * 32 < c.n_parts) d += v[u];
    }
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (threadIdx.x == 0) {
      const float f = (float)d, sc = (float)c.scale, top = (float)c.max_norm, eps = (float)c.eps;
      float norm = fabsf(sc) * sqrtf(f), coef = top / (norm + eps), by;
      if (f > 1e-24f && f < 1e36f && norm > 1e-12f && norm < 1e18f && top > 1e-12f && top < 1e18f && eps < 1e18f) {
        coef = coef >= 1.f ? 1.f : coef;
        by = sc * coef;
      } else {
        const double nd = fabs(c.scale) * sqrt(d), r = c.max_norm / (nd + c.eps), cd = r >= 1.0 ? 1.0 : r;     // NaN stays
        norm = (float)nd;
        coef = (float)cd;
        by = (float)(c.scale * cd);
      }
      if (write) {
        c.stats[0] = norm;
        if (c.clip) c.stats[1] = coef;
      }
      factor = by;
    }
  }
  __syncthreads();
  return factor;
}
__global__ void __launch_bounds__(32) norm_k(Clip c) {
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
  // The two never reach a boundary together: by element, clipping 219M of fp32 takes 1080
  // us instead of 405, of bf16 952 instead of 207.
  if (head != gc_head(o, n)) {
    for (long long i = threadIdx.x; i < n; i += GC_THREADS) o[i] = gc_t<T>(gc_f(p[i]) * f);
    return;
  }
  if ((int)threadIdx.x < head) o[threadIdx.x] = gc_t<T>(gc_f(p[threadIdx.x]) * f);
  const long long vecs = (n - head) / 8;
  const int tail = (int)(n - head - vecs * 8);
  p += head;
  o += head;
  if ((int)threadIdx.x < tail) o[vecs * 8 + threadIdx.x] = gc_t<T>(gc_f(p[vecs * 8 + threadIdx.x]) * f);
  // from the end: what the squares read last is the likeliest to be in L2 still
  for (long long i = vecs - 1 - threadIdx.x; i >= 0; i -= GC_FLIGHT * GC_THREADS) {
    Raw8<T> v[GC_FLIGHT];
#pragma unroll
    for (int u = 0; u < GC_FLIGHT; ++u)
      if (i - u * GC_THREADS >= 0) v[u].template load<2>(p + (i - u * GC_THREADS) * 8, 0, 8);
#pragma unroll
    for (int u = 0; u < GC_FLIGHT; ++u) {
      if (i - u * GC_THREADS < 0) break;
      float x[8];
      v[u].values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f;
      ops_st8<2>(o + (i - u * GC_THREADS) * 8, 0, 8, x);
    }
  }
}

// The same runs, from their ends.  876 MB of fp32 into as many: 270 us, 95 % of the copy
// rate; a unit to each CTA in turn instead of a run takes as long there, and 45 us
// instead of 26 for 500 ragged tensors.
template <int N>
__global__ void __launch_bounds__(GC_THREADS, GC_CTAS) scale_k(const __grid_constant__ Table<N> t, Clip c, int first) {
  ops_begin();
  const float f = gc_factor(c, first && blockIdx.x == 0);
  const uint32_t units = t.start[t.n], begin = gc_share(units, blockIdx.x);
  uint32_t u = gc_share(units, blockIdx.x + 1);
  if (u <= begin) return;
  for (int s = gc_find(t, u - 1); u > begin; --s) {
    const uint32_t from = t.start[s], low = from > begin ? from : begin;
    if (low >= u) continue;
    const long long lo = (long long)(low - from) * GC_UNIT, to = (long long)(u - from) * GC_UNIT;
    const long long n = (to < t.numel[s] ? to : t.numel[s]) - lo;
    u = low;
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
  const uint32_t most = (uint32_t)ops_least(GC_CTAS * sms, GC_PARTS);
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
  if (!ops_device(&dev, &sms)) return MT_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  c.parts = (const double*)ws;
  c.n_parts = 0;
  for (int i = 0; i < n; i += GC_TABLE) {
    int used = 0;
    const int rc = launch_any(s + i, ops_least(n - i, GC_TABLE), sms, (double*)ws + c.n_parts, nullptr, 0, &used, st);
    if (rc) return rc;
    c.n_parts += used;
  }
  if (!c.clip || n == 0) return ops_launch(norm_k, 1, 32, 0, st, 1, c);
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
