// block_norm.cu - the joint between two blocks (mt_block_norm) and its gradients
// (mt_block_norm_bwd): norm after a block, gate, scaled residual sum, norm
// before the next block.
#include <math.h>
#include <string.h>

#include "ops8.cuh"

namespace {

#define BN_MAX_WIDTH 8192
#define BN_MAX_PARTS 256          // CTAs that leave partial column sums

struct Joint {
  const float *after, *before;
  const void* gate;
  long long ldgate;
  const int* n_rows;
  int rows, width, gate_kind;
  float a, b, eps;
};
struct Fwd {
  Joint j;
  const void *x, *y;
  void *h, *r;
  long long ldx, ldy, ldh, ldr;
};
struct Bwd {
  Joint j;
  const void *h, *y, *dr, *dh;
  void *dx, *dy, *dgate;
  long long ldh, ldy, lddr, lddh, lddx, lddy, lddgate;
  float* ws;                      // [CTAs][sums][width]: dbefore, dafter, dgate where there are such sums
};

// Columns of a lane within a chunk of 256: eight neighbours, or (no alignment)
// every 32nd, so that neighbouring lanes take neighbouring elements.
template <int VEC>
__device__ __forceinline__ int bn_col(int chunk, int lane) {
  return chunk * 256 + (VEC ? lane * 8 : lane);
}
// VEC: rows are whole eights on their boundaries, a lane's eight lie inside or outside
template <int VEC, class T>
__device__ __forceinline__ void bn_load(Raw8<T>& v, const T* p, int c, int n) {
  if (!VEC || c < n) v.template load<VEC ? 2 : 0, 32>(p, c, n);
  else memset(&v, 0, sizeof(v));
}
template <int VEC>
__device__ __forceinline__ void bn_vec(const float* p, int c, int n, float* v) {
  if (!VEC || c < n) {
    ops_ld8<VEC ? 2 : 0, 32>(p, c, n, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
}
template <int VEC, class T>
__device__ __forceinline__ void bn_store(T* p, int c, int n, const float* v) {
  if (!VEC || c < n) ops_st8<VEC ? 2 : 0, 32>(p, c, n, v);
}
__device__ __forceinline__ float bn_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One pass over the rows: x and y are read once, kept in registers (8 C columns
// per lane) over the two sums of squares, and h and r written once.  Up to 1024
// columns a warp takes a row and nothing is shared; wider rows take a CTA of as
// many warps as they have 1024 columns.
template <class S, class T, int VEC, int C, bool WIDE>
__global__ void __launch_bounds__(256) block_norm_k(Fwd f) {
  ops_begin();
  __shared__ float red[2][8];
  const Joint& j = f.j;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = WIDE ? (int)blockDim.x >> 5 : 1;
  const int first = WIDE ? warp : 0, n = j.width;
  const long long row = WIDE ? (long long)blockIdx.x : (long long)blockIdx.x * 8 + warp;
  if (row >= ops_row_limit(j.n_rows, j.rows)) return;
  const float mean = 1.f / (float)n;
  Raw8<S> xs[C];
  Raw8<T> ys[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = bn_col<VEC>(first + i * warps, lane);
    bn_load<VEC>(xs[i], (const S*)f.x + row * f.ldx, c, n);
    if (f.y) bn_load<VEC>(ys[i], (const T*)f.y + row * f.ldy, c, n);
  }
  float inv = 1.f;
  if (j.after) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
      ys[i].values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
    }
    s = bn_sum(s);
    if (WIDE) {
      if (lane == 0) red[0][warp] = s;
      __syncthreads();
      s = 0.f;
      for (int w = 0; w < warps; ++w) s += red[0][w];
    }
    inv = __frsqrt_rn(fmaf(s, mean, j.eps));
  }
  const float by = j.gate_kind == MT_GATE_TOKEN ? ((const float*)j.gate)[row * j.ldgate] * j.b : j.b;
  float h[C][8], s = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = bn_col<VEC>(first + i * warps, lane);
    xs[i].values(h[i]);
    if (f.y) {
      float v[8], g[8];
      ys[i].values(v);
      if (j.after) {
        bn_vec<VEC>(j.after, c, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * g[e];
      }
      if (j.gate_kind == MT_GATE_CHANNEL) {
        bn_vec<VEC>((const float*)j.gate, c, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= g[e];
      } else if (j.gate_kind == MT_GATE_FULL) {
        Raw8<T> gt;
        bn_load<VEC>(gt, (const T*)j.gate + row * j.ldgate, c, n);
        gt.values(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = fmaf(j.a, h[i][e], by * v[e]);
      bn_store<VEC>((S*)f.h + row * f.ldh, c, n, h[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(h[i][e], h[i][e], s);
  }
  if (!j.before) return;
  s = bn_sum(s);
  if (WIDE) {
    if (lane == 0) red[1][warp] = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[1][w];
  }
  inv = __frsqrt_rn(fmaf(s, mean, j.eps));
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = bn_col<VEC>(first + i * warps, lane);
    float g[8];
    bn_vec<VEC>(j.before, c, n, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = h[i][e] * inv * g[e];
    bn_store<VEC>((T*)f.r + row * f.ldr, c, n, g);
  }
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// Sums of K values over a group of `warps` warps (named barrier `bar`); every
// lane gets them.  red: two buffers of the group, taken in turn: whoever writes one
// again has passed the other's barrier, and with it every warp's reads of this one.
template <int K>
__device__ __forceinline__ void bn_group_sum(float (&s)[K], float* red, int warps, int w, int lane, int bar, int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = bn_sum(s[k]);
  if (warps == 1) return;
  red += turn * warps * 4;
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) red[w * K + k] = s[k];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * warps) : "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = 0.f;
  for (int i = 0; i < warps; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += red[i * K + k];
  }
}

template <class S, class T>
struct BwdRow {
  Raw8<S> h, dh;
  Raw8<T> dr, y, gate;
};
template <int VEC, class S, class T>
__device__ __forceinline__ void bn_row(BwdRow<S, T>& v, const Bwd& f, long long row, int c) {
  const int n = f.j.width;
  if (f.dh) bn_load<VEC>(v.dh, (const S*)f.dh + row * f.lddh, c, n);
  if (f.j.before) {
    bn_load<VEC>(v.h, (const S*)f.h + row * f.ldh, c, n);
    bn_load<VEC>(v.dr, (const T*)f.dr + row * f.lddr, c, n);
  }
  if (f.y) bn_load<VEC>(v.y, (const T*)f.y + row * f.ldy, c, n);
  if (f.j.gate_kind == MT_GATE_FULL) bn_load<VEC>(v.gate, (const T*)f.j.gate + row * f.j.ldgate, c, n);
}

// Persistent CTAs of G groups; a group of W warps takes a row, a lane 8 C fixed
// columns of it, so the gains and the column sums stay in registers from row to
// row.  With rh = 1 / rms(h), u = dr * before:
//   G = dh + rh u - h rh^3 mean(u h)          dx = a G, dbefore += dr h rh
//   g = b G, n = y ry after, v = g gate       dgate += g n, dafter += v y ry
//   dy = ry w - y ry^3 mean(w y), w = v after
// Two sums over the row: (h^2, u h, y^2), then (w y, g n).  The next row is on
// its way while this one is computed (C 1).
template <class S, class T, int VEC, int C>
__global__ void __launch_bounds__(512, 1) block_norm_bwd_k(Bwd f, int W, int G) {
  ops_begin();
  extern __shared__ float sh[];
  const Joint& j = f.j;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = wid / W, w = wid - g * W, n = j.width;
  float* red = sh + g * W * 8;              // two buffers of four values per warp
  int turn = 0;
  const int bar = 1 + g;
  const int lim = ops_row_limit(j.n_rows, j.rows), step = (int)gridDim.x * G;
  const float mean = 1.f / (float)n;
  const bool channel = j.gate_kind == MT_GATE_CHANNEL, token = j.gate_kind == MT_GATE_TOKEN,
             full = j.gate_kind == MT_GATE_FULL;
  float kb[C][8], ka[C][8], kg[C][8], sb[C][8], sa[C][8], sg[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = bn_col<VEC>(w + i * W, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) kb[i][e] = ka[i][e] = kg[i][e] = 1.f, sb[i][e] = sa[i][e] = sg[i][e] = 0.f;
    if (j.before) bn_vec<VEC>(j.before, c, n, kb[i]);
    if (j.after) bn_vec<VEC>(j.after, c, n, ka[i]);
    if (channel) bn_vec<VEC>((const float*)j.gate, c, n, kg[i]);
  }
  BwdRow<S, T> cur[C];
  long long row = (long long)blockIdx.x * G + g;
  if (C == 1 && row < lim) bn_row<VEC>(cur[0], f, row, bn_col<VEC>(w, lane));
  for (; row < lim; row += step) {
    BwdRow<S, T> next;
    if (C > 1) {
#pragma unroll
      for (int i = 0; i < C; ++i) bn_row<VEC>(cur[i], f, row, bn_col<VEC>(w + i * W, lane));
    } else if (row + step < lim) {
      bn_row<VEC>(next, f, row + step, bn_col<VEC>(w, lane));
    }
    const float tg = token ? ((const float*)j.gate)[row * j.ldgate] : 1.f;
    float s1[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float h[8], v[8];
      if (j.before) {
        cur[i].h.values(h);
        cur[i].dr.values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s1[0] = fmaf(h[e], h[e], s1[0]);
          s1[1] = fmaf(v[e] * kb[i][e], h[e], s1[1]);
        }
      }
      if (j.after) {
        cur[i].y.values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s1[2] = fmaf(v[e], v[e], s1[2]);
      }
    }
    bn_group_sum(s1, red, W, w, lane, bar, turn);
    const float rh = j.before ? __frsqrt_rn(fmaf(s1[0], mean, j.eps)) : 0.f;
    const float ry = j.after ? __frsqrt_rn(fmaf(s1[2], mean, j.eps)) : 1.f;
    const float qh = rh * rh * rh * (s1[1] * mean);
    float s2[2] = {0.f, 0.f}, gr[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = bn_col<VEC>(w + i * W, lane);
      float h[8], v[8], o[8];
      if (f.dh) cur[i].dh.values(gr[i]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) gr[i][e] = 0.f;
      if (j.before) {
        cur[i].h.values(h);
        cur[i].dr.values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = v[e] * rh;
          sb[i][e] = fmaf(t, h[e], sb[i][e]);
          gr[i][e] += fmaf(t, kb[i][e], -h[e] * qh);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = j.a * gr[i][e];
      bn_store<VEC>((S*)f.dx + row * f.lddx, c, n, o);
      if (!f.y) continue;
      cur[i].y.values(v);
      float gt[8];
      if (full) cur[i].gate.values(gt);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = j.b * gr[i][e], yn = v[e] * ry, gn = t * (yn * ka[i][e]);
        if (channel) sg[i][e] += gn;
        if (token) s2[1] += gn;
        if (full) o[e] = gn;
        const float u = t * (full ? gt[e] : channel ? kg[i][e] : tg);
        sa[i][e] = fmaf(u, yn, sa[i][e]);
        gr[i][e] = u * ka[i][e];
        s2[0] = fmaf(gr[i][e], v[e], s2[0]);
      }
      if (full) bn_store<VEC>((T*)f.dgate + row * f.lddgate, c, n, o);
    }
    if (f.y) {
      if (j.after || token) bn_group_sum(s2, red, W, w, lane, bar, turn);
      if (token && w == 0 && lane == 0) ((float*)f.dgate)[row * f.lddgate] = s2[1];
      const float qy = j.after ? ry * ry * ry * (s2[0] * mean) : 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float v[8];
        cur[i].y.values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(gr[i][e], ry, -v[e] * qy);
        bn_store<VEC>((T*)f.dy + row * f.lddy, bn_col<VEC>(w + i * W, lane), n, v);
      }
    }
    if (C == 1) cur[0] = next;
  }
  // the groups' column sums, in the groups' order
  const int nb = j.before ? 1 : 0, na = j.after ? 1 : 0, ns = nb + na + (channel ? 1 : 0);
  if (!ns) return;
  float* part = f.ws + (long long)blockIdx.x * ns * n;
  float* to = G > 1 ? sh : part;
  for (int gg = 0; gg < G; ++gg) {
    __syncthreads();                        // the row sums' buffers, then the group before
    if (g != gg) continue;
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k == 0 ? !nb : k == 1 ? !na : !channel) continue;
        const float* v = k == 0 ? sb[i] : k == 1 ? sa[i] : sg[i];
        float* p = to + (long long)(k == 0 ? 0 : k == 1 ? nb : nb + na) * n;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = bn_col<VEC>(w + i * W, lane) + (VEC ? e : 32 * e);
          if (c < n) p[c] = gg ? p[c] + v[e] : v[e];
        }
      }
    }
  }
  if (G == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < ns * n; c += blockDim.x) part[c] = sh[c];
}

// Column sums of the CTAs' parts: eight warps take every eighth part of 32
// columns, joined in order.
struct Sums {
  const float* ws;
  float* out[3];
  int parts, width, sums, accumulate;
};
__global__ void __launch_bounds__(256) column_sums_k(Sums s) {
  ops_begin();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, k = blockIdx.y;
  const long long step = (long long)s.sums * s.width;
  float v = 0.f;
  constexpr int U = 20;                       // all in flight: 152 parts by eight warps
  for (int p0 = w; p0 < s.parts && c < s.width; p0 += 8 * U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = p0 + 8 * u < s.parts ? s.ws[(p0 + 8 * u) * step + (long long)k * s.width + c] : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) v += x[u];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w || c >= s.width) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += red[i][lane];
  float* out = k == 0 ? s.out[0] : k == 1 ? s.out[1] : s.out[2];
  out[c] = s.accumulate ? out[c] + v : v;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int joint_ok(const mt_joint* j) {
  if (!j || j->reserved0 || j->rows < 0 || j->width < 1) return MT_ERR_ARG;
  if (!ops_dtype_ok(j->stream_dtype) || !ops_dtype_ok(j->dtype)) return MT_ERR_ARG;
  if (j->rows > OPS_MAX_ROWS || j->width > BN_MAX_WIDTH) return MT_ERR_UNSUPPORTED;
  if (j->stream_dtype == MT_DT_BF16 && j->dtype == MT_DT_FP32) return MT_ERR_UNSUPPORTED;
  if (!(j->eps > 0.f) || isinf(j->eps) || !isfinite(j->res_scale) || !isfinite(j->out_scale)) return MT_ERR_ARG;
  if (j->gate_kind < MT_GATE_NONE || j->gate_kind > MT_GATE_FULL) return MT_ERR_ARG;
  if ((j->gate != nullptr) != (j->gate_kind != MT_GATE_NONE)) return MT_ERR_ARG;
  if (!ops_aligned(j->after, 4) || !ops_aligned(j->before, 4) || !ops_aligned(j->n_rows, 4)) return MT_ERR_ARG;
  if (j->gate_kind == MT_GATE_CHANNEL && !ops_aligned(j->gate, 4)) return MT_ERR_ARG;
  if (j->gate_kind == MT_GATE_TOKEN && !ops_mat_ok(j->gate, MT_DT_FP32, j->ldgate, 1)) return MT_ERR_ARG;
  if (j->gate_kind == MT_GATE_FULL && !ops_mat_ok(j->gate, j->dtype, j->ldgate, j->width)) return MT_ERR_ARG;
  return MT_OK;
}
Joint joint(const mt_joint* j) {
  return {j->after, j->before, j->gate, (long long)j->ldgate, j->n_rows, (int)j->rows, (int)j->width, j->gate_kind,
          j->res_scale, j->out_scale, j->eps};
}
// whole eights everywhere: columns, rows' starts, gains
bool joint_vec(const mt_joint* j) {
  return j->width % 8 == 0 && ops_aligned(j->after, 32) && ops_aligned(j->before, 32) &&
         (j->gate_kind != MT_GATE_CHANNEL || ops_aligned(j->gate, 32)) &&
         (j->gate_kind != MT_GATE_FULL || ops_vec(j->gate, j->dtype, j->ldgate) == 2);
}
bool mat_vec(const void* p, int dtype, int64_t ld) { return !p || ops_vec(p, dtype, ld) == 2; }

template <class S, class T, int VEC>
int fwd_t(const Fwd& f, cudaStream_t st) {
  const int chunks = (f.j.width + 255) / 256;
  if (chunks <= 4) {
    auto k = chunks == 1   ? block_norm_k<S, T, VEC, 1, false>
             : chunks == 2 ? block_norm_k<S, T, VEC, 2, false>
             : chunks == 3 ? block_norm_k<S, T, VEC, 3, false>
                           : block_norm_k<S, T, VEC, 4, false>;
    return ops_launch(k, (unsigned)((f.j.rows + 7) / 8), 256, 0, st, 1, f);
  }
  return ops_launch(block_norm_k<S, T, VEC, 4, true>, (unsigned)f.j.rows, 32u * (unsigned)((chunks + 3) / 4), 0, st, 1, f);
}

// warps of a row, and rows at once of a CTA of up to 16 warps
int bwd_warps(int64_t width) {
  const int chunks = (int)((width + 255) / 256);
  return chunks <= 16 ? chunks : (chunks + 1) / 2;
}
template <class S, class T, int VEC>
int bwd_t(const Bwd& f, int sms, int* parts, cudaStream_t st) {
  const int W = bwd_warps(f.j.width), most = ops_least(sms, BN_MAX_PARTS);
  // rows are spread over the CTAs before any takes two at once
  const int per = (f.j.rows + most - 1) / most, G = ops_least(16 / W, per);
  *parts = ops_least((f.j.rows + G - 1) / G, most);
  size_t smem = (size_t)G * W * 8 * 4, sums = G > 1 ? (size_t)3 * f.j.width * 4 : 0;
  if (smem < sums) smem = sums;
  auto k = W * 256 >= f.j.width ? block_norm_bwd_k<S, T, VEC, 1> : block_norm_bwd_k<S, T, VEC, 2>;
  return ops_launch(k, (unsigned)*parts, 32u * W * G, smem, st, 1, f, W, G);
}

}  // namespace

extern "C" {

int32_t mt_block_norm(const mt_joint* j, const void* x, int64_t ldx, const void* y, int64_t ldy, void* h, int64_t ldh,
                      void* r, int64_t ldr, void* stream) {
  const int st = joint_ok(j);
  if (st) return st;
  if (j->rows == 0) return MT_OK;
  // y brings h, `before` brings r, and something has to be made
  if ((y != nullptr) != (h != nullptr) || (j->before != nullptr) != (r != nullptr) || (!h && !r)) return MT_ERR_ARG;
  if (!y && (j->after || j->gate || j->res_scale != 1.f)) return MT_ERR_ARG;
  if (!ops_mat_ok(x, j->stream_dtype, ldx, j->width)) return MT_ERR_ARG;
  if (y && (!ops_mat_ok(y, j->dtype, ldy, j->width) || !ops_mat_ok(h, j->stream_dtype, ldh, j->width))) return MT_ERR_ARG;
  if (r && !ops_mat_ok(r, j->dtype, ldr, j->width)) return MT_ERR_ARG;
  const bool vec = joint_vec(j) && mat_vec(x, j->stream_dtype, ldx) && mat_vec(y, j->dtype, ldy) &&
                   mat_vec(h, j->stream_dtype, ldh) && mat_vec(r, j->dtype, ldr);
  const Fwd f = {joint(j), x, y, h, r, ldx, ldy, ldh, ldr};
  cudaStream_t s = (cudaStream_t)stream;
  if (j->stream_dtype == MT_DT_BF16) return vec ? fwd_t<__nv_bfloat16, __nv_bfloat16, 1>(f, s) : fwd_t<__nv_bfloat16, __nv_bfloat16, 0>(f, s);
  if (j->dtype == MT_DT_BF16) return vec ? fwd_t<float, __nv_bfloat16, 1>(f, s) : fwd_t<float, __nv_bfloat16, 0>(f, s);
  return vec ? fwd_t<float, float, 1>(f, s) : fwd_t<float, float, 0>(f, s);
}

int64_t mt_block_norm_ws_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || width < 1) return -MT_ERR_ARG;
  if (rows > OPS_MAX_ROWS || width > BN_MAX_WIDTH) return -MT_ERR_UNSUPPORTED;
  return (rows < 1 ? 1 : rows < BN_MAX_PARTS ? rows : BN_MAX_PARTS) * 3 * width * 4;
}

int32_t mt_block_norm_bwd(const mt_joint* j, const void* h, int64_t ldh, const void* y, int64_t ldy, const void* dr,
                          int64_t lddr, const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dy, int64_t lddy,
                          void* dgate, int64_t lddgate, float* dafter, float* dbefore, int32_t accumulate, void* ws,
                          int64_t ws_bytes, void* stream) {
  const int st = joint_ok(j);
  if (st) return st;
  const bool channel = j->gate_kind == MT_GATE_CHANNEL;
  if (accumulate != 0 && accumulate != 1) return MT_ERR_ARG;
  if ((j->after != nullptr) != (dafter != nullptr) || (j->before != nullptr) != (dbefore != nullptr) ||
      !ops_aligned(dafter, 4) || !ops_aligned(dbefore, 4))
    return MT_ERR_ARG;
  if (channel && (!dgate || !ops_aligned(dgate, 4))) return MT_ERR_ARG;
  if (j->rows) {
    const int sd = j->stream_dtype, od = j->dtype;
    const int64_t n = j->width;
    if ((y != nullptr) != (dy != nullptr) || (j->gate != nullptr) != (dgate != nullptr) || (!dr && !dh)) return MT_ERR_ARG;
    if ((j->before != nullptr) != (dr != nullptr)) return MT_ERR_ARG;
    if (!y && (j->after || j->gate || j->res_scale != 1.f)) return MT_ERR_ARG;
    if (!ops_mat_ok(dx, sd, lddx, n) || (dh && !ops_mat_ok(dh, sd, lddh, n))) return MT_ERR_ARG;
    if (dr && (!ops_mat_ok(dr, od, lddr, n) || !ops_mat_ok(h, sd, ldh, n))) return MT_ERR_ARG;
    if (y && (!ops_mat_ok(y, od, ldy, n) || !ops_mat_ok(dy, od, lddy, n))) return MT_ERR_ARG;
    if (j->gate_kind == MT_GATE_TOKEN && !ops_mat_ok(dgate, MT_DT_FP32, lddgate, 1)) return MT_ERR_ARG;
    if (j->gate_kind == MT_GATE_FULL && !ops_mat_ok(dgate, od, lddgate, n)) return MT_ERR_ARG;
  }
  const int sums = (dbefore ? 1 : 0) + (dafter ? 1 : 0) + (channel ? 1 : 0);
  if (sums && (!ws || !ops_aligned(ws, 16))) return MT_ERR_ARG;
  if (sums && ws_bytes < mt_block_norm_ws_bytes(j->rows, j->width)) return MT_ERR_ARENA_SMALL;
  cudaStream_t s = (cudaStream_t)stream;
  int parts = 0;
  if (j->rows) {
    int dev, sms;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return MT_ERR_CUDA;
    }
    const Bwd f = {joint(j), dr ? h : nullptr, y, dr, dh, dx, dy, dgate, ldh, ldy, lddr, lddh, lddx, lddy, lddgate, (float*)ws};
    const bool vec = joint_vec(j) && mat_vec(f.h, j->stream_dtype, ldh) && mat_vec(y, j->dtype, ldy) &&
                     mat_vec(dr, j->dtype, lddr) && mat_vec(dh, j->stream_dtype, lddh) &&
                     mat_vec(dx, j->stream_dtype, lddx) && mat_vec(dy, j->dtype, lddy) &&
                     (j->gate_kind != MT_GATE_FULL || mat_vec(dgate, j->dtype, lddgate));
    auto k = j->stream_dtype == MT_DT_BF16 ? (vec ? bwd_t<__nv_bfloat16, __nv_bfloat16, 1> : bwd_t<__nv_bfloat16, __nv_bfloat16, 0>)
             : j->dtype == MT_DT_BF16      ? (vec ? bwd_t<float, __nv_bfloat16, 1> : bwd_t<float, __nv_bfloat16, 0>)
                                           : (vec ? bwd_t<float, float, 1> : bwd_t<float, float, 0>);
    const int rc = k(f, sms, &parts, s);
    if (rc) return rc;
  }
  if (!sums) return MT_OK;
  Sums c = {(const float*)ws, {}, parts, (int)j->width, sums, accumulate};
  int k = 0;
  if (dbefore) c.out[k++] = dbefore;
  if (dafter) c.out[k++] = dafter;
  if (channel) c.out[k++] = (float*)dgate;
  return ops_launch(column_sums_k, dim3((unsigned)((j->width + 31) / 32), (unsigned)sums), 256, 0, s, 1, c);
}

}  // extern "C"
