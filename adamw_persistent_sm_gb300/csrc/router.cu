// router.cu - the choice of experts from the router's logits with counts and
// losses (mt_choose), and the gradient for the logits (mt_choose_bwd).
#include <float.h>
#include <math.h>

#include "ops8.cuh"

namespace {

#define RT_E MT_MAX_EXPERTS
#define RT_K 8
#define RT_WARPS 28              // of a CTA that takes tiles of 32 rows
#define RT_TILES 300000          // choices from which tiles are taken
// CTAs that leave parts: for each expert the sum of its probabilities, the sum of
// squared logs, then the counts and the number of tokens
#define RT_MAX_PARTS 152

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
  const float many = tokens > 0 ? (float)tokens : 1.f;
  float s = 0.f;
  for (int e = lane; e < c.E; e += 32) {
    s = fmaf((float)n[e] / many, p[e] / many, s);
    c.counts[e] = n[e];
  }
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane) return;
  c.counts[c.E] = tokens;
  c.losses[0] = s * ((float)c.E / (float)c.K);
  c.losses[1] = size / many;
}
__device__ __forceinline__ void rt_order(float& a, float& b) {
  const float t = fminf(a, b);
  a = fmaxf(a, b);
  b = t;
}
// The eight largest values of a row so far, descending; take8 adds eight more.
struct Top8 {
  float v[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = -INFINITY;
  }
  // Batcher's network of 19 exchanges sorts the eight; the larger of v[i] and
  // z[7 - i] are the eight largest of both, and rise once and fall once: three
  // more stages sort them.
  __device__ __forceinline__ void take8(float* z) {
    rt_order(z[0], z[1]); rt_order(z[2], z[3]); rt_order(z[4], z[5]); rt_order(z[6], z[7]);
    rt_order(z[0], z[2]); rt_order(z[1], z[3]); rt_order(z[4], z[6]); rt_order(z[5], z[7]);
    rt_order(z[1], z[2]); rt_order(z[5], z[6]);
    rt_order(z[0], z[4]); rt_order(z[1], z[5]); rt_order(z[2], z[6]); rt_order(z[3], z[7]);
    rt_order(z[2], z[4]); rt_order(z[3], z[5]);
    rt_order(z[1], z[2]); rt_order(z[3], z[4]); rt_order(z[5], z[6]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaxf(v[i], z[7 - i]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & o)) rt_order(v[i], v[i + o]);
  }
  // how many are larger than z, which at least one is not
  __device__ __forceinline__ int larger(float z) const {
    const bool four = v[3] > z, two = (four ? v[5] : v[1]) > z;
    const bool one = (four ? (two ? v[6] : v[4]) : (two ? v[2] : v[0])) > z;
    return four * 4 + two * 2 + one;
  }
};
// eight words, of which the first four lie at p + at and the others at p + (at ^ 4)
__device__ __forceinline__ void rt_get8(const float* p, int at, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + (at ^ 4));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void rt_put8(float* p, int at, const float* v) {
  *reinterpret_cast<float4*>(p + at) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + (at ^ 4)) = make_float4(v[4], v[5], v[6], v[7]);
}
// e^(z - top), 0 for -inf; off by 2 ulp and |z - top| / 2 more
__device__ __forceinline__ float rt_exp(float z, float top) {
  float x;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"((z - top) * 1.4426950408889634f));
  return x;
}

// Few tokens, or few choices of each: L lanes share a row, V logits each, and a warp
// takes 32 / L rows at a time.  The maximum, the sum of exponentials and the K
// choices (the largest left over, the lowest expert among equals) stay in registers;
// probabilities are summed by expert over the warp's rows in registers too, and
// joined by warp, CTA and part in a fixed order.  Launches and their latency bound it:
// 2.6 us for a token, 6.0 for 32,768 with 2 of 16 experts (2.6 MB), of which the join
// takes 1.5 to 2; 1,024 tokens in one CTA took 11, spread over many with a join 4.4.
// 131,072 tokens take 10.4 us, with 4 of 16 13.4: a warp's next rows are not on their way
// while it chooses, and each choice is a search over the lanes of a row.
template <class Z, int V, int L, int KM, bool VEC>
__global__ void __launch_bounds__(1024) choose_lanes_k(Choose c) {
  ops_begin();
  __shared__ float p_warp[32][RT_E], s_warp[32];
  __shared__ int hist[RT_E], t_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, l = lane & (L - 1);
  for (int e = threadIdx.x; e < RT_E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  float psum[V] = {}, size = 0.f;
  int tokens = 0;
  const long long step = (long long)gridDim.x * warps * (32 / L);
  for (long long r0 = ((long long)warp * gridDim.x + blockIdx.x) * (32 / L); r0 < c.tokens; r0 += step) {
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
      p[v] = open ? rt_exp(z[v], top) : 0.f;
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
    float best[KM], total = 0.f;
    int at[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
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
      best[k] = take ? rt_exp(b, top) : 0.f;
      at[k] = take ? e : -1;
      total += best[k];
    }
    const float scale = bad && live ? NAN : !open ? 0.f : c.renormalize ? 1.f / total : inv;
#pragma unroll
    for (int k = 0; k < KM; ++k) {
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
    for (int i = 0; i < warps; ++i) s += p_warp[i][threadIdx.x];
    p_warp[0][threadIdx.x] = s;
  }
  __syncthreads();
  if (warp) return;
  size = 0.f;
  tokens = 0;
  for (int i = 0; i < warps; ++i) {
    size += s_warp[i];
    tokens += t_warp[i];
  }
  if (gridDim.x == 1) {
    rt_finish(c, p_warp[0], hist, size, tokens);
    return;
  }
  uint32_t* part = c.ws + (long long)blockIdx.x * (2 * c.E + 2);
  for (int e = lane; e < c.E; e += 32) {
    part[e] = __float_as_uint(p_warp[0][e]);
    part[c.E + 1 + e] = (uint32_t)hist[e];
  }
  if (lane == 0) {
    part[c.E] = __float_as_uint(size);
    part[2 * c.E + 1] = (uint32_t)tokens;
  }
}

// Many choices: a warp takes 32 rows at a time through its part of shared memory: they come in
// whole lines, then a lane has a row of its own - the eight largest by a sorting
// network (two instructions an exchange for 32 rows), the bits of the logits that
// reach the K-th, whose places follow from how many of the sorted values are larger,
// and the sum of exponentials - and last a lane has an expert (PAIR: two), whose
// probabilities it sums over the 32 rows and on.  All in a fixed order, as are
// warps, CTAs and parts.  16-byte piece p of row r lies at p ^ r: accesses of 16
// bytes by rows and of words by experts meet no bank twice, and 28 warps fit an SM.
// 131,072 tokens, 8 of 64 experts, bf16: 24 us, lanes 43.  The time of one warp's tile
// bounds it, from its loads to its last sum: 65,536 tokens, the same tiles on half the
// warps, take 24 us too, though at 131,072 the issue slots are 60 % used (the pipe of
// comparisons 54 %).  Some 110 instructions a row, of which the network takes 17 (by
// lanes that share a row it would take 80).  With rows 68 words apart instead, 24 warps
// to an SM and a second round for an eighth of them: 27 us; that round all in the first
// CTAs: 43.
template <class Z, bool VEC, bool PAIR>
__global__ void __launch_bounds__(32 * RT_WARPS) choose_tiles_k(Choose c) {
  ops_begin();
  extern __shared__ __align__(16) float sh[];
  __shared__ float s_warp[RT_WARPS];
  __shared__ int hist[RT_E], t_warp[RT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = c.E, K = c.K;
  constexpr int LD = PAIR ? 64 : 32, KM = RT_K;            // words of a row
  float* tile = sh + warp * 32 * LD;
  float* mine = tile + lane * LD;
  const int sw = (lane & (LD / 4 - 1)) * 4;                // word e of this lane's row is at e ^ sw
  for (int e = threadIdx.x; e < RT_E; e += blockDim.x) hist[e] = 0;
  const int up = (E + 7) & ~7;
  for (int e = E; e < up; ++e) mine[e ^ sw] = -INFINITY;   // up to whole eights
  __syncthreads();
  float sum[2] = {0.f, 0.f}, size = 0.f;
  int tokens = 0;
  constexpr int CH = VEC ? 16 / (int)sizeof(Z) : 1;        // elements of a load
  const int per = E / CH;                                  // loads of a row
  const uint32_t inv_per = ((1u << 20) + per - 1) / per;   // i / per for i < 2048: i * (per - 1) < 2^20
  // a round of tiles goes over all CTAs before any takes more
  const long long step = (long long)gridDim.x * warps * 32;
  for (long long r0 = ((long long)warp * gridDim.x + blockIdx.x) * 32; r0 < c.tokens; r0 += step) {
    const int rows = c.tokens - r0 < 32 ? (int)(c.tokens - r0) : 32;
    const Z* z0 = (const Z*)c.z + r0 * c.ldz;
    if constexpr (VEC) {
      constexpr int U = 4;
      for (int i0 = lane; i0 < rows * per; i0 += 32 * U) {
        uint4 u[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = i0 + 32 * k, r = (int)((uint32_t)i * inv_per >> 20);
          if (i < rows * per) u[k] = *reinterpret_cast<const uint4*>(z0 + r * c.ldz + (i - r * per) * CH);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = i0 + 32 * k, r = (int)((uint32_t)i * inv_per >> 20);
          if (i >= rows * per) break;
          const int to = r * LD + ((i - r * per) * CH ^ (r & (LD / 4 - 1)) * 4);
          if constexpr (CH == 4) {
            *reinterpret_cast<uint4*>(tile + to) = u[k];
          } else {
            *reinterpret_cast<float4*>(tile + to) = make_float4(ops_lo(u[k].x), ops_hi(u[k].x), ops_lo(u[k].y), ops_hi(u[k].y));
            *reinterpret_cast<float4*>(tile + (to ^ 4)) = make_float4(ops_lo(u[k].z), ops_hi(u[k].z), ops_lo(u[k].w), ops_hi(u[k].w));
          }
        }
      }
    } else {
      for (int i = lane; i < rows * E; i += 32) {
        const int r = (int)((uint32_t)i * inv_per >> 20), e = i - r * E;
        tile[r * LD + (e ^ (r & (LD / 4 - 1)) * 4)] = (float)z0[r * c.ldz + e];
      }
    }
    const long long row = r0 + lane;
    const bool there = lane < rows;
    bool live = there && (!c.mask || c.mask[row]);
    __syncwarp();
    Top8 top;
    top.clear();
    for (int e0 = 0; e0 < E; e0 += 8) {
      float z[8];
      rt_get8(mine, e0 ^ sw, z);
      top.take8(z);
    }
    float kth = top.v[0];
#pragma unroll
    for (int k = 1; k < KM; ++k) kth = k < K ? top.v[k] : kth;
    const float m = top.v[0] > -INFINITY ? top.v[0] : 0.f;
    uint32_t reach[2] = {0, 0};
    for (int e0 = 0; e0 < E; e0 += 8) {
      uint32_t b = 0;
      float z[8];
      rt_get8(mine, e0 ^ sw, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) b |= z[i] >= kth ? 1u << i : 0u;
      if (e0 < 32) reach[0] |= b << e0;
      else reach[1] |= b << (e0 - 32);
    }
    if (!(kth > -INFINITY)) {                     // fewer than K experts are open: only those
      reach[0] = reach[1] = 0;
      for (int e = 0; e < E; ++e)
        if (mine[e ^ sw] > -INFINITY) reach[e >> 5] |= 1u << (e & 31);
    }
    if (!live) reach[0] = reach[1] = 0;
    uint32_t at[2] = {~0u, ~0u}, used = 0;        // a byte per place
    for (int half = 0; half < (PAIR ? 2 : 1); ++half) {
      for (uint32_t left = reach[half]; __any_sync(0xffffffffu, left); left &= left - 1) {
        const int e = __ffs(left) - 1 + 32 * half;
        if (left) {
          int k = top.larger(mine[e ^ sw]);
          k += __ffs(~(used >> k)) - 1;             // equals in the order of their experts
          if (k < K) {
            used |= 1u << k;
            at[k >> 2] ^= (uint32_t)(0xff ^ e) << (8 * (k & 3));
          }
        }
      }
    }
    // exponentials in place of the logits; a row that holds NaN or +inf, which the
    // values above do not show, has a sum that is NaN
    float s = 0.f;
    for (int e0 = 0; e0 < E; e0 += 8) {
      float z[8];
      rt_get8(mine, e0 ^ sw, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = rt_exp(z[i], m);
      s += ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
      rt_put8(mine, e0 ^ sw, z);
    }
    const bool bad = live && !(s <= FLT_MAX);
    live = live && s != 0.f;
    const bool open = live && !bad;
    const float inv = open ? 1.f / s : bad ? NAN : 0.f;
    if (live) {
      const float lse = bad ? NAN : m + logf(s);
      size = fmaf(lse, lse, size);
      ++tokens;
    } else {
      for (int e = 0; e < E; ++e) mine[e ^ sw] = 0.f;
    }
    float w[KM], total = 0.f;
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      w[k] = k < K && open ? rt_exp(top.v[k], m) : 0.f;
      total += w[k];
    }
    const float by = !open ? inv : c.renormalize ? 1.f / total : inv;
    __syncwarp();
#pragma unroll 8
    for (int r = 0; r < rows; ++r) {
      const float iv = __shfl_sync(0xffffffffu, inv, r);
      if constexpr (PAIR) {
        const float2 x = *reinterpret_cast<const float2*>(tile + r * LD + (2 * lane ^ (r & 15) * 4));
        sum[0] = fmaf(x.x, iv, sum[0]);
        sum[1] = fmaf(x.y, iv, sum[1]);
      } else {
        sum[0] = fmaf(tile[r * LD + (lane ^ (r & 7) * 4)], iv, sum[0]);
      }
    }
    __syncwarp();
    // the choices leave in whole lines, through the tile; 17 and 9 words to a row of it
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      if (k >= K) break;
      const int e = open ? at[k >> 2] >> (8 * (k & 3)) & 0xff : 0xff;
      tile[lane * (2 * KM + 1) + k] = __int_as_float(e == 0xff ? -1 : e);
      tile[lane * (2 * KM + 1) + KM + k] = w[k] * by;
      if (e != 0xff) atomicAdd(&hist[e], 1);
    }
    __syncwarp();
    const uint32_t inv_k = ((1u << 16) + K - 1) / K;       // i / K for i < 256
    for (int i = lane; i < rows * K; i += 32) {
      const int r = (int)((uint32_t)i * inv_k >> 16), at_ = r * (2 * KM + 1) + i - r * K;
      c.idx[r0 * K + i] = __float_as_int(tile[at_]);
      c.w[r0 * K + i] = tile[at_ + KM];
    }
    __syncwarp();
    for (int e = E; e < up; ++e) mine[e ^ sw] = -INFINITY;
  }
  // the tiles are done with: each warp's sums in its own
#pragma unroll
  for (int i = 0; i < (PAIR ? 2 : 1); ++i) tile[PAIR ? 2 * lane + i : lane] = sum[i];
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
  if (warp) return;
  for (int e = lane; e < E; e += 32) {
    float a = 0.f;
    for (int i = 0; i < warps; ++i) a += sh[i * 32 * LD + e];
    sh[e] = a;
  }
  __syncwarp();
  size = 0.f;
  tokens = 0;
  for (int i = 0; i < warps; ++i) {
    size += s_warp[i];
    tokens += t_warp[i];
  }
  if (gridDim.x == 1) {
    rt_finish(c, sh, hist, size, tokens);
    return;
  }
  uint32_t* part = c.ws + (long long)blockIdx.x * (2 * E + 2);
  for (int e = lane; e < E; e += 32) {
    part[e] = __float_as_uint(sh[e]);
    part[E + 1 + e] = (uint32_t)hist[e];
  }
  if (lane == 0) {
    part[E] = __float_as_uint(size);
    part[2 * E + 1] = (uint32_t)tokens;
  }
}

// The parts joined: `wide` threads (whole warps) take a word each, of every
// slices-th part, thirteen loads on their way at once: all of 152 parts up to 31
// experts, which have sixteen slices (16 experts: 1.5 to 2 us, one load after the other
// 5).  32 experts have ten and 64 six, and take two rounds.
__global__ void __launch_bounds__(1024) choose_join_k(Choose c, int parts, int wide) {
  ops_begin();
  __shared__ float p[RT_E + 1];
  __shared__ int n[RT_E + 1];
  __shared__ uint32_t red[1024];
  const int words = 2 * c.E + 2, i = threadIdx.x % wide, s = threadIdx.x / wide, slices = blockDim.x / wide;
  const bool real = i <= c.E;
  float a = 0.f;
  int b = 0;
  constexpr int U = 13;
  for (int k0 = s; k0 < parts && i < words; k0 += U * slices) {
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = k0 + u * slices < parts ? __ldcg(c.ws + (long long)(k0 + u * slices) * words + i) : 0u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (real) a += __uint_as_float(v[u]);
      else b += (int)v[u];
    }
  }
  red[threadIdx.x] = real ? __float_as_uint(a) : (uint32_t)b;
  __syncthreads();
  if (s == 0 && i < words) {
    for (int k = 1; k < slices; ++k) {
      const uint32_t v = red[k * wide + i];
      if (real) a += __uint_as_float(v);
      else b += (int)v;
    }
    if (real) p[i] = a;
    else n[i - c.E - 1] = b;
  }
  __syncthreads();
  if (threadIdx.x < 32) rt_finish(c, p, n, p[c.E], n[c.E]);
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
// Logits of -inf, which also stand for experts that there are not and for tokens that
// take no part, neither take a dw nor get a gradient: by selection, for an infinite
// factor times their probability of 0 is NaN.
// 3.7 to 4.1 us for 32,768 tokens with 16 experts (4.7 MB): its launch and latency.
// 131,072 tokens: 10 us, and 32 with 8 of 64 experts, fp32 or bf16 (11 and 6 by bytes):
// every lane of a row reads all its indices and their gradients.
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
        if (rt_expert<V, L, VEC>(l, v) == e && z[v] > -INFINITY) {
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
  for (int v = 0; v < V; ++v) o[v] = bad && live ? NAN : z[v] > -INFINITY ? o[v] : 0.f;
  if (there) rt_store<Z, V, L, VEC>((Z*)c.dz + row * c.lddz, l, c.E, o);
}

int choose_ok(int64_t tokens, int32_t K, int32_t E, int32_t dtype, int64_t ldz, const void* mask, int32_t renormalize) {
  if (tokens < 0 || K < 1 || E < 1 || !ops_dtype_ok(dtype) || (renormalize != 0 && renormalize != 1)) return MT_ERR_ARG;
  if (E > RT_E || K > RT_K || K > E || tokens > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  return MT_OK;
}
int lanes_of(int E) { return E <= 8 ? 2 : E <= 16 ? 4 : 8; }
// a lane's logits lie on their own boundary: E is a multiple of the 4 (8) of a lane
bool rows_vec(const void* z, int dtype, int64_t ld, int E) {
  const int V = E <= 32 ? 4 : 8, B = ops_least(V * ops_size(dtype), 16);
  return E % V == 0 && ops_aligned(z, B) && ld * ops_size(dtype) % B == 0;
}

// What a call launches: warps of a CTA, CTAs and the kernel.
struct Plan {
  int warps;
  int64_t parts;
  bool tiles;
};
Plan choose_plan(int64_t tokens, int K, int E) {
  Plan p;
  // Lanes against tiles, us at 65,536 / 131,072 tokens: 3 of 64 experts 16.4 / 25.2
  // against 19.8 / 19.9, 8 of 64 25.5 / 43.1 against 22.4 / 22.3, 8 of 32 20.4 / 33.7
  // against 16.0 / 16.0, 6 of 24 16.8 / 27.2 against 14.1 / 14.4; at 32,768 lanes
  // win everywhere (8 of 64: 16.0 against 18.2), and with 16 experts (4: 13.3
  // against 14.7) or two choices at every size.
  p.tiles = K > 2 && E > 16 && tokens * K > RT_TILES;
  const int rows = p.tiles ? 32 : 32 / lanes_of(E), most = p.tiles ? RT_WARPS : 32;       // of a warp; warps of a CTA
  const int64_t units = (tokens + rows - 1) / rows, w = (units + RT_MAX_PARTS - 1) / RT_MAX_PARTS;
  // sixteen warps in one CTA need no join; more spread over CTAs of at least four
  const bool alone = units <= 16;
  p.warps = alone ? (units < 1 ? 1 : (int)units) : w < 4 ? 4 : w < most ? (int)w : most;
  const int64_t n = alone ? 1 : (units + p.warps - 1) / p.warps;
  p.parts = n < RT_MAX_PARTS ? n : RT_MAX_PARTS;
  return p;
}
template <class Z, bool VEC>
int choose_t(const Choose& c, const Plan& plan, cudaStream_t st) {
  int rc;
  if (plan.tiles) {
    const size_t smem = (size_t)plan.warps * 32 * (c.E <= 32 ? 32 : 64) * 4;
    auto k = c.E <= 32 ? choose_tiles_k<Z, VEC, false> : choose_tiles_k<Z, VEC, true>;
    int dev, sms;
    if (!ops_device(&dev, &sms)) return MT_ERR_CUDA;
    rc = ops_launch_wide(k, dev, (size_t)RT_WARPS * 8192, (unsigned)plan.parts, 32u * plan.warps, smem, st, c);
  } else {
    auto k = c.K <= 2 ? (c.E <= 8    ? choose_lanes_k<Z, 4, 2, 2, VEC>
                         : c.E <= 16 ? choose_lanes_k<Z, 4, 4, 2, VEC>
                         : c.E <= 32 ? choose_lanes_k<Z, 4, 8, 2, VEC>
                                     : choose_lanes_k<Z, 8, 8, 2, VEC>)
                      : (c.E <= 8    ? choose_lanes_k<Z, 4, 2, 8, VEC>
                         : c.E <= 16 ? choose_lanes_k<Z, 4, 4, 8, VEC>
                         : c.E <= 32 ? choose_lanes_k<Z, 4, 8, 8, VEC>
                                     : choose_lanes_k<Z, 8, 8, 8, VEC>);
    rc = ops_launch(k, (unsigned)plan.parts, 32u * plan.warps, 0, st, 1, c);
  }
  if (rc || plan.parts == 1) return rc;
  const int wide = (2 * c.E + 2 + 31) / 32 * 32;
  return ops_launch(choose_join_k, 1, (unsigned)(1024 / wide * wide), 0, st, 1, c, (int)plan.parts, wide);
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
  return (choose_plan(n_tokens, top_k, n_experts).parts * (2 * n_experts + 2) * 4 + 15) / 16 * 16;
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
  const Plan plan = choose_plan(n_tokens, top_k, n_experts);
  const int whole = 16 / ops_size(dtype);
  const bool vec = plan.tiles ? n_experts % whole == 0 && ops_aligned(logits, 16) && ldz % whole == 0
                              : rows_vec(logits, dtype, ldz, n_experts);
  auto f = dtype == MT_DT_FP32 ? (vec ? choose_t<float, true> : choose_t<float, false>)
                               : (vec ? choose_t<__nv_bfloat16, true> : choose_t<__nv_bfloat16, false>);
  return f(c, plan, (cudaStream_t)stream);
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
