// router.cu - the choice of experts from the router's logits with counts and
// losses (mt_choose), and the gradient for the logits (mt_choose_bwd).
#include <float.h>
#include <math.h>

#include "ops8.cuh"

namespace {

#define RT_E MT_MAX_EXPERTS
#define RT_K 8
#define RT_THREADS 512
#define RT_MAX_PARTS 304          // CTAs that leave partial sums
// words of a CTA's part: probabilities summed by expert, counts, then the sum of
// squared logs and the number of tokens
#define RT_PART (2 * RT_E + 2)

// Experts of lane l of the L that share a row: V neighbours, or every L-th.
template <int V, int L, bool VEC>
__device__ __forceinline__ int rt_expert(int l, int v) {
  return VEC ? l * V + v : v * L + l;
}
// Logits of a lane, -inf where there is no expert.  -0 becomes 0, so that equal
// values are equal.
template <class Z, int V, int L, bool VEC>
__device__ __forceinline__ void rt_load(const Z* z, int l, int E, float* v) {
  if constexpr (VEC) {
    constexpr int B = V * (int)sizeof(Z);          // 8, 16 or 32 bytes
    uint32_t u[B / 4];
    if (l * V < E) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(z + l * V);
#pragma unroll
      for (int i = 0; i < B / 4; i += (B >= 16 ? 4 : 2)) {
        if constexpr (B >= 16) {
          const uint4 q = *reinterpret_cast<const uint4*>(p + i);
          u[i] = q.x; u[i + 1] = q.y; u[i + 2] = q.z; u[i + 3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(p + i);
          u[i] = q.x; u[i + 1] = q.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float x;
      if constexpr (sizeof(Z) == 4) x = __uint_as_float(u[i]);
      else x = i & 1 ? ops_hi(u[i / 2]) : ops_lo(u[i / 2]);
      v[i] = l * V < E ? x + 0.f : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * L + l;
      v[i] = e < E ? (float)z[e] + 0.f : -INFINITY;
    }
  }
}
template <class Z, int V, int L, bool VEC>
__device__ __forceinline__ void rt_store(Z* z, int l, int E, const float* v) {
  if constexpr (VEC) {
    if (l * V >= E) return;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if constexpr (sizeof(Z) == 4) *reinterpret_cast<float4*>(z + l * V + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      else *reinterpret_cast<uint2*>(z + l * V + i) = make_uint2(ops_bf2(v[i], v[i + 1]), ops_bf2(v[i + 2], v[i + 3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * L + l < E) z[i * L + l] = (Z)v[i];
  }
}
template <int L>
__device__ __forceinline__ float rt_sum(float s) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
template <int L>
__device__ __forceinline__ float rt_max(float s) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
  return s;
}
// whether any lane of the row says so
template <int L>
__device__ __forceinline__ bool rt_any(bool b) {
  const uint32_t all = __ballot_sync(0xffffffffu, b);
  return all >> ((threadIdx.x & 31) & ~(L - 1)) & (L == 32 ? 0xffffffffu : (1u << L) - 1);
}

struct Choose {
  const void* z;
  const uint8_t* mask;
  int* idx;
  float* w;
  int* counts;
  float* losses;
  uint32_t* ws;
  long long ldz, tokens;
  int E, K, renormalize;
};

// The losses from the totals, by the first warp: f_e = counts_e / (K N), P_e =
// sum of probabilities / N, balance = E sum f_e P_e; and the mean squared log.
__device__ void rt_finish(const Choose& c, const float* p, const int* n, float size, int tokens) {
  const int lane = threadIdx.x & 31;
  const double many = tokens > 0 ? (double)tokens : 1.0;
  double s = 0.0;
  for (int e = lane; e < c.E; e += 32) {
    s += (double)n[e] * (double)p[e];
    c.counts[e] = n[e];
  }
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane) return;
  c.counts[c.E] = tokens;
  c.losses[0] = (float)(s * (double)c.E / ((double)c.K * many * many));
  c.losses[1] = (float)((double)size / many);
}

// L lanes share a row, V logits each; a warp takes 32 / L rows at a time.  The
// maximum, the sum of exponentials and the K choices (the largest left over, the
// lowest expert among equals) stay in registers; probabilities are summed by
// expert over the warp's rows in registers too, and joined by warp, CTA and part
// in a fixed order.
template <class Z, int V, int L, bool VEC>
__global__ void __launch_bounds__(RT_THREADS) choose_k(Choose c) {
  ops_begin();
  constexpr int WARPS = RT_THREADS / 32;
  __shared__ float p_warp[WARPS][RT_E], s_warp[WARPS];
  __shared__ int hist[RT_E], t_warp[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1);
  for (int e = threadIdx.x; e < RT_E; e += RT_THREADS) hist[e] = 0;
  __syncthreads();
  float psum[V] = {}, size = 0.f;
  int tokens = 0;
  const long long step = (long long)gridDim.x * (RT_THREADS / L);
  for (long long r0 = ((long long)blockIdx.x * WARPS + warp) * (32 / L); r0 < c.tokens; r0 += step) {
    const long long row = r0 + lane / L;
    const bool there = row < c.tokens;
    float z[V], p[V];
    bool live = there && (!c.mask || c.mask[row]);
    if (live) rt_load<Z, V, L, VEC>((const Z*)c.z + row * c.ldz, l, c.E, z);
    else
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = -INFINITY;
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m = fmaxf(m, z[v]);
      bad |= !(z[v] <= FLT_MAX);
    }
    m = rt_max<L>(m);
    bad = rt_any<L>(bad);
    live = live && (bad || m > -INFINITY);
    const bool open = live && !bad;
    const float top = open ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = open ? expf(z[v] - top) : 0.f;
      s += p[v];
    }
    s = rt_sum<L>(s);
    const float inv = open ? 1.f / s : bad ? NAN : 0.f;
    if (live) {
      const float lse = bad ? NAN : top + logf(s);
      size += l == 0 ? lse * lse : 0.f;
      tokens += l == 0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (live) psum[v] += p[v] * inv;
    float best[RT_K], total = 0.f;
    int at[RT_K];
#pragma unroll
    for (int k = 0; k < RT_K; ++k) {
      if (k >= c.K) break;
      float b = -INFINITY;
      int e = RT_E;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (z[v] > b) {
          b = z[v];
          e = rt_expert<V, L, VEC>(l, v);
        }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, b, o);
        const int oe = __shfl_xor_sync(0xffffffffu, e, o);
        if (ob > b || (ob == b && oe < e)) {
          b = ob;
          e = oe;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (rt_expert<V, L, VEC>(l, v) == e) z[v] = -INFINITY;
      const bool take = open && b > -INFINITY;
      best[k] = take ? expf(b - top) : 0.f;
      at[k] = take ? e : -1;
      total += best[k];
    }
    const float scale = bad && live ? NAN : !open ? 0.f : c.renormalize ? 1.f / total : inv;
#pragma unroll
    for (int k = 0; k < RT_K; ++k) {
      if (k >= c.K) break;
      if ((k & (L - 1)) != l || !there) continue;
      c.idx[row * c.K + k] = at[k];
      c.w[row * c.K + k] = best[k] * scale;
      if (at[k] >= 0) atomicAdd(&hist[at[k]], 1);
    }
  }
  // the warp's rows, then the CTA's warps
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) psum[v] += __shfl_xor_sync(0xffffffffu, psum[v], o);
    if (lane < L) p_warp[warp][rt_expert<V, L, VEC>(l, v)] = psum[v];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    size += __shfl_xor_sync(0xffffffffu, size, o);
    tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
  }
  if (lane == 0) {
    s_warp[warp] = size;
    t_warp[warp] = tokens;
  }
  __syncthreads();
  if (threadIdx.x < V * L) {
    float s = 0.f;
    for (int i = 0; i < WARPS; ++i) s += p_warp[i][threadIdx.x];
    p_warp[0][threadIdx.x] = s;
  }
  __syncthreads();
  if (warp) return;
  size = 0.f;
  tokens = 0;
  for (int i = 0; i < WARPS; ++i) {
    size += s_warp[i];
    tokens += t_warp[i];
  }
  if (gridDim.x == 1) {
    rt_finish(c, p_warp[0], hist, size, tokens);
    return;
  }
  uint32_t* part = c.ws + (long long)blockIdx.x * RT_PART;
  for (int e = lane; e < c.E; e += 32) {
    part[e] = __float_as_uint(p_warp[0][e]);
    part[RT_E + e] = (uint32_t)hist[e];
  }
  if (lane == 0) {
    part[2 * RT_E] = __float_as_uint(size);
    part[2 * RT_E + 1] = (uint32_t)tokens;
  }
}

// The parts joined: a thread takes every eighth part of one word.
__global__ void __launch_bounds__(1024) choose_join_k(Choose c, int parts) {
  ops_begin();
  __shared__ float p[8][RT_E + 1];
  __shared__ int n[8][RT_E + 1];
  const int e = threadIdx.x & 127, s = threadIdx.x >> 7;          // 128 words, eight slices
  if (e <= RT_E) {
    const bool last = e == RT_E;
    float a = 0.f;
    int b = 0;
    if (last || e < c.E) {
#pragma unroll 8
      for (int i = s; i < parts; i += 8) {
        const uint32_t* part = c.ws + (long long)i * RT_PART;
        a += __uint_as_float(part[last ? 2 * RT_E : e]);
        b += (int)part[last ? 2 * RT_E + 1 : RT_E + e];
      }
    }
    p[s][e] = a;
    n[s][e] = b;
  }
  __syncthreads();
  if (threadIdx.x <= RT_E) {
    float a = 0.f;
    int b = 0;
    for (int i = 0; i < 8; ++i) {
      a += p[i][threadIdx.x];
      b += n[i][threadIdx.x];
    }
    p[0][threadIdx.x] = a;
    n[0][threadIdx.x] = b;
  }
  __syncthreads();
  if (threadIdx.x < 32) rt_finish(c, p[0], n[0], p[0][RT_E], n[0][RT_E]);
}

struct ChooseBwd {
  const void* z;
  const uint8_t* mask;
  const int* idx;
  const int* counts;
  const float* dw;
  const float* dlosses;
  void* dz;
  long long ldz, lddz, tokens;
  int E, K, renormalize;
};

// The same rows and lanes.  With p the probabilities, w the weights of the chosen:
//   weights  chosen j: w_j (dw_j - sum w dw); without renormalising p_j (dw_j - sum p dw), for every j
//   balance  E / (K N^2) p_j (counts_j - sum_e counts_e p_e)
//   size     2 / N lse p_j
template <class Z, int V, int L, bool VEC>
__global__ void __launch_bounds__(256) choose_bwd_k(ChooseBwd c) {
  ops_begin();
  const int lane = threadIdx.x & 31, l = lane & (L - 1);
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / L;
  const bool there = row < c.tokens;
  bool live = there && (!c.mask || c.mask[row]);
  float z[V];
  if (live) rt_load<Z, V, L, VEC>((const Z*)c.z + row * c.ldz, l, c.E, z);
  else
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = -INFINITY;
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m = fmaxf(m, z[v]);
    bad |= !(z[v] <= FLT_MAX);
  }
  m = rt_max<L>(m);
  bad = rt_any<L>(bad);
  live = live && (bad || m > -INFINITY);
  const bool open = live && !bad;
  const float top = open ? m : 0.f;
  float ex[V], d[V] = {}, s = 0.f, load = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ex[v] = open ? expf(z[v] - top) : 0.f;
    s += ex[v];
  }
  s = rt_sum<L>(s);
  const float inv = open ? 1.f / s : 0.f;
  float o[V] = {};
  if (c.dw) {
    uint32_t chosen = 0;
    for (int k = 0; k < c.K; ++k) {
      const int e = there ? c.idx[row * c.K + k] : -1;
      const float dk = there && e >= 0 ? c.dw[row * c.K + k] : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (rt_expert<V, L, VEC>(l, v) == e) {
          d[v] += dk;
          chosen |= 1u << v;
        }
    }
    float total = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (chosen >> v & 1) {
        total += ex[v];
        dot = fmaf(ex[v], d[v], dot);
      }
    dot = rt_sum<L>(dot);
    total = rt_sum<L>(total);
    const float scale = c.renormalize ? (total > 0.f ? 1.f / total : 0.f) : inv;
    dot *= scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool part = !c.renormalize || (chosen >> v & 1);
      o[v] = part ? ex[v] * scale * (d[v] - dot) : 0.f;
    }
  }
  if (c.dlosses) {
    const int n = c.counts[c.E];
    const float many = n > 0 ? (float)n : 1.f;
    const float c0 = c.dlosses[0] * (float)c.E / ((float)c.K * many * many), c1 = c.dlosses[1] * 2.f / many;
    const float lse = open ? top + logf(s) : 0.f;
    float cnt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = rt_expert<V, L, VEC>(l, v);
      cnt[v] = e < c.E ? (float)c.counts[e] : 0.f;
      load = fmaf(ex[v] * inv, cnt[v], load);
    }
    load = rt_sum<L>(load);
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] += ex[v] * inv * (c0 * (cnt[v] - load) + c1 * lse);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = bad && live ? NAN : o[v];
  if (there) rt_store<Z, V, L, VEC>((Z*)c.dz + row * c.lddz, l, c.E, o);
}

int choose_ok(int64_t tokens, int32_t K, int32_t E, int32_t dtype, int64_t ldz, const void* mask, int32_t renormalize) {
  if (tokens < 0 || K < 1 || E < 1 || !ops_dtype_ok(dtype) || (renormalize != 0 && renormalize != 1)) return MT_ERR_ARG;
  if (E > RT_E || K > RT_K || K > E || tokens > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  return MT_OK;
}
int64_t choose_parts(int64_t tokens, int lanes) {
  const int64_t n = (tokens + RT_THREADS / lanes - 1) / (RT_THREADS / lanes);
  return n < 1 ? 1 : n < RT_MAX_PARTS ? n : RT_MAX_PARTS;
}
int lanes_of(int E) { return E <= 8 ? 2 : E <= 16 ? 4 : 8; }
// a lane's logits lie on their own boundary: E is a multiple of the 4 (8) of a lane
bool rows_vec(const void* z, int dtype, int64_t ld, int E) {
  const int V = E <= 32 ? 4 : 8, B = ops_least(V * ops_size(dtype), 16);
  return E % V == 0 && ops_aligned(z, B) && ld * ops_size(dtype) % B == 0;
}

template <class Z, bool VEC>
int choose_t(const Choose& c, cudaStream_t st) {
  const int lanes = lanes_of(c.E);
  const unsigned parts = (unsigned)choose_parts(c.tokens, lanes);
  auto k = c.E <= 8    ? choose_k<Z, 4, 2, VEC>
           : c.E <= 16 ? choose_k<Z, 4, 4, VEC>
           : c.E <= 32 ? choose_k<Z, 4, 8, VEC>
                       : choose_k<Z, 8, 8, VEC>;
  const int rc = ops_launch(k, parts, RT_THREADS, 0, st, 1, c);
  return rc || parts == 1 ? rc : ops_launch(choose_join_k, 1, 1024, 0, st, 1, c, (int)parts);
}
template <class Z, bool VEC>
int choose_bwd_t(const ChooseBwd& c, cudaStream_t st) {
  const unsigned grid = (unsigned)((c.tokens * lanes_of(c.E) + 255) / 256);
  auto k = c.E <= 8    ? choose_bwd_k<Z, 4, 2, VEC>
           : c.E <= 16 ? choose_bwd_k<Z, 4, 4, VEC>
           : c.E <= 32 ? choose_bwd_k<Z, 4, 8, VEC>
                       : choose_bwd_k<Z, 8, 8, VEC>;
  return ops_launch(k, grid, 256, 0, st, 1, c);
}

}  // namespace

extern "C" {

int64_t mt_choose_ws_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts) {
  const int st = choose_ok(n_tokens, top_k, n_experts, MT_DT_FP32, 0, nullptr, 0);
  if (st) return -st;
  return choose_parts(n_tokens, lanes_of(n_experts)) * RT_PART * 4;
}

int32_t mt_choose(const void* logits, int32_t dtype, int64_t ldz, int64_t n_tokens, int32_t n_experts, int32_t top_k,
                  const uint8_t* mask, int32_t renormalize, int32_t* idx, float* w, int32_t* counts, float* losses,
                  void* ws, int64_t ws_bytes, void* stream) {
  const int st = choose_ok(n_tokens, top_k, n_experts, dtype, ldz, mask, renormalize);
  if (st) return st;
  if (!counts || !losses || !ops_aligned(counts, 4) || !ops_aligned(losses, 4)) return MT_ERR_ARG;
  if (n_tokens && (!idx || !w || !ops_aligned(idx, 4) || !ops_aligned(w, 4) || !ops_mat_ok(logits, dtype, ldz, n_experts)))
    return MT_ERR_ARG;
  if (!ws || !ops_aligned(ws, 16)) return MT_ERR_ARG;
  if (ws_bytes < mt_choose_ws_bytes(n_tokens, top_k, n_experts)) return MT_ERR_ARENA_SMALL;
  const Choose c = {logits, mask, idx, w, counts, losses, (uint32_t*)ws, ldz, n_tokens, n_experts, top_k, renormalize};
  const bool vec = rows_vec(logits, dtype, ldz, n_experts);
  auto f = dtype == MT_DT_FP32 ? (vec ? choose_t<float, true> : choose_t<float, false>)
                               : (vec ? choose_t<__nv_bfloat16, true> : choose_t<__nv_bfloat16, false>);
  return f(c, (cudaStream_t)stream);
}

int32_t mt_choose_bwd(const void* logits, int32_t dtype, int64_t ldz, int64_t n_tokens, int32_t n_experts,
                      int32_t top_k, const uint8_t* mask, int32_t renormalize, const int32_t* idx,
                      const int32_t* counts, const float* dw, const float* dlosses, void* dlogits, int64_t lddz,
                      void* stream) {
  const int st = choose_ok(n_tokens, top_k, n_experts, dtype, ldz, mask, renormalize);
  if (st) return st;
  if (n_tokens == 0) return MT_OK;
  if (!dw && !dlosses) return MT_ERR_ARG;
  if (dlosses && (!counts || !ops_aligned(counts, 4) || !ops_aligned(dlosses, 4))) return MT_ERR_ARG;
  if (dw && (!idx || !ops_aligned(idx, 4) || !ops_aligned(dw, 4))) return MT_ERR_ARG;
  if (!ops_mat_ok(logits, dtype, ldz, n_experts) || !ops_mat_ok(dlogits, dtype, lddz, n_experts)) return MT_ERR_ARG;
  const ChooseBwd c = {logits, mask, idx, counts, dw, dlosses, dlogits, ldz, lddz, n_tokens, n_experts, top_k, renormalize};
  const bool vec = rows_vec(logits, dtype, ldz, n_experts) && rows_vec(dlogits, dtype, lddz, n_experts);
  auto f = dtype == MT_DT_FP32 ? (vec ? choose_bwd_t<float, true> : choose_bwd_t<float, false>)
                               : (vec ? choose_bwd_t<__nv_bfloat16, true> : choose_bwd_t<__nv_bfloat16, false>);
  return f(c, (cudaStream_t)stream);
}

}  // extern "C"
