// quant8.cu - matrices into 8 bits and back (mt_quant8, mt_quant8_t,
// mt_dequant8) and the SwiGLU that keeps its inputs there (mt_swiglu8,
// mt_swiglu8_bwd).
#include <string.h>

#include "ops8.cuh"

namespace {

struct Mat8 {
  uint8_t* q;
  uint8_t* s;
  long long ld, lds;
  int rows, cols;
};
Mat8 mat8(const mt_mat8* m) {
  return {(uint8_t*)m->codes, (uint8_t*)m->scales, m->ld, m->lds, (int)m->rows, (int)m->cols};
}

// ---------------------------------------------------------------------------
// 1 x 128 blocks along the rows
// ---------------------------------------------------------------------------
// A half warp holds one block in registers (8 elements per lane): its maximum
// is four shuffles, x is read once and the codes are written once.  A warp
// takes R rows of the same 256 columns and issues all their loads first.
// Columns come in `parts` of `pcols` with blocks of their own.
template <class T, int VEC, int R>
__global__ void __launch_bounds__(256) quant_rows_k(const T* x, long long ldx, const int* n_rows, Mat8 o, int parts,
                                                    int pcols) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lim = ops_row_limit(n_rows, o.rows);
  const int r0 = ((int)blockIdx.x * 8 + warp) * R;
  if (r0 >= lim) return;
  const int chunks = (pcols + 255) / 256, pblocks = (pcols + 127) / 128;
  const bool v8 = (pcols & 7) == 0;
  for (int ch = blockIdx.y; ch < parts * chunks; ch += gridDim.y) {
    const int part = ch / chunks, c = (ch - part * chunks) * 256 + lane * 8, base = part * pcols;
    Raw8<T> x8[R];
    uint32_t top[R];
    // rows past the limit repeat the last one, and are not stored
#pragma unroll
    for (int i = 0; i < R; ++i) x8[i].template load<VEC>(x + (long long)min(r0 + i, lim - 1) * ldx + base, c, pcols);
#pragma unroll
    for (int i = 0; i < R; ++i) top[i] = x8[i].top();
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r0 + i >= lim) break;
      float v[8];
      uint32_t e;
      x8[i].values(v);
      const uint2 q = ops_quantise(v, top[i], &e);
      ops_st_codes<VEC>(o.q + (long long)(r0 + i) * o.ld + base, c, pcols, q, v8 || parts == 1);
      if ((lane & 15) == 0 && c < pcols) o.s[(long long)(r0 + i) * o.lds + part * pblocks + (c >> 7)] = (uint8_t)e;
    }
  }
}

template <class T, int VEC>
__global__ void __launch_bounds__(256) dequant_k(Mat8 a, const int* n_rows, int parts, int pcols, T* out,
                                                 long long ldo) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lim = ops_row_limit(n_rows, a.rows);
  const int r0 = ((int)blockIdx.x * 8 + warp) * 4;
  if (r0 >= lim) return;
  const int chunks = (pcols + 255) / 256, pblocks = (pcols + 127) / 128;
  const bool v8 = (pcols & 7) == 0 || parts == 1;
  for (int ch = blockIdx.y; ch < parts * chunks; ch += gridDim.y) {
    const int part = ch / chunks, c = (ch - part * chunks) * 256 + lane * 8, base = part * pcols;
    if (c >= pcols) continue;
    uint2 q[4];
    uint32_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = min(r0 + i, lim - 1);
      q[i] = ops_ld_codes<VEC>(a.q + r * a.ld + base, c, pcols, v8);
      s[i] = a.s[r * a.lds + part * pblocks + (c >> 7)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < lim) {
        float v[8];
        ops_values8(q[i], ops_byte_scale(s[i]), v);
        ops_st8<VEC>(out + (long long)(r0 + i) * ldo + base, c, pcols, v);
      }
  }
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles: blocks of 128 x 128, straight or transposed, and
// transposed 1 x 128 blocks (128 rows of one column)
// ---------------------------------------------------------------------------
enum { T_BLOCK = 0, T_BLOCK_T = 1, T_COLS_T = 2 };

// Eight elements of a row of an 8-bit matrix, kept as codes and scale.
struct Src8 {
  const uint8_t* q;
  const uint8_t* s;
  long long ld, lds;
};
struct RawCodes {
  uint2 q;
  float s;
  __device__ __forceinline__ void values(float* v) const { ops_values8(q, s, v); }
};
template <class T>
struct Tile8 {
  typedef Raw8<T> Raw;
  template <int VEC>
  static __device__ __forceinline__ void load(Raw& w, const T* x, long long ldx, const Src8&, long long r, int c,
                                              int n) {
    w.template load<VEC>(x + r * ldx, c, n);
  }
  static __device__ __forceinline__ void zero(Raw& w) { memset(&w, 0, sizeof(w)); }
};
template <>
struct Tile8<uint8_t> {
  typedef RawCodes Raw;
  template <int VEC>
  static __device__ __forceinline__ void load(Raw& w, const uint8_t*, long long, const Src8& a, long long r,
                                              int c, int n) {
    w.q = make_uint2(0, 0);
    w.s = 1.f;
    if (VEC != 2 && c >= n) return;
    w.q = ops_ld_codes<VEC>(a.q + r * a.ld, c, n, true);
    w.s = ops_byte_scale(a.s[r * a.lds + (c >> 7)]);
  }
  static __device__ __forceinline__ void zero(Raw& w) {
    w.q = make_uint2(0, 0);
    w.s = 1.f;
  }
};
// bits of the largest magnitude in each of the eight columns over eight rows
__device__ __forceinline__ void tile_top(const Raw8<__nv_bfloat16>* w, uint32_t* m) {
  uint32_t a[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].u.x, w[i].u.y, w[i].u.z, w[i].u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = ops_max_u16x2(a[j], u[j] & 0x7fff7fffu);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[2 * j] = a[j] << 16;
    m[2 * j + 1] = a[j] & 0xffff0000u;
  }
}
template <class RAW>
__device__ __forceinline__ void tile_top(const RAW* w, uint32_t* m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    w[i].values(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = max(m[j], __float_as_uint(v[j]) & 0x7fffffffu);
  }
}

// A thread holds 8 rows x 8 columns of a tile as they came from memory.  A column's
// maximum goes over 8 rows in registers, two lanes by shuffle and 8 warps through
// shared memory; transposed codes go through a 16 KB tile whose 8-byte chunks are
// swizzled by the source column group, which keeps both sides free of bank
// conflicts.  Memory-bound: each byte is read and written once.  A CTA walks over
// tiles, columns fastest, and (PRE) reads the next while it converts one.
template <class T, int VEC, int MODE>
__global__ void __launch_bounds__(256, sizeof(T) == 1 ? 3 : 2) quant_tile_k(const T* x, long long ldx, Src8 src, const int* n_rows, Mat8 o,
                                                       int rows, int cols) {
  // fp32: two tiles would not fit the registers; codes: bound by their conversions,
  // three CTAs without reading ahead take 30 us where two that do take 35
  constexpr bool PRE = sizeof(T) == 2;
  __shared__ uint32_t part[8][128];
  __shared__ float inv[128];
  __shared__ __align__(16) uint2 tile[MODE == T_BLOCK ? 1 : 128 * 16];
  ops_begin();
  typedef typename Tile8<T>::Raw Raw;
  const int tid = threadIdx.x, warp = tid >> 5, tc = tid & 15, tr = tid >> 4;
  const int b = blockIdx.z, nct = (cols + 127) / 128;
  const int lim = ops_row_limit(n_rows, rows);
  const long long tiles = (long long)((lim + 127) / 128) * nct;
  const T* xb = x + (long long)b * rows * ldx;
  auto load = [&](Raw* w, long long t) {
    const int rt = (int)(t / nct), r0 = rt * 128 + tr * 8, c0 = (int)(t - (long long)rt * nct) * 128 + tc * 8;
    if (rt * 128 + 128 <= lim) {
#pragma unroll
      for (int i = 0; i < 8; ++i) Tile8<T>::template load<VEC>(w[i], xb, ldx, src, r0 + i, c0, cols);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i < lim) Tile8<T>::template load<VEC>(w[i], xb, ldx, src, r0 + i, c0, cols);
        else Tile8<T>::zero(w[i]);
      }
    }
  };
  Raw next[8];
  if (PRE && blockIdx.x < tiles) load(next, blockIdx.x);
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    {
      const int rt = (int)(t / nct), ct = (int)(t - (long long)rt * nct);
      const int r0 = rt * 128 + tr * 8, c0 = ct * 128 + tc * 8;
      Raw w[8];
      if (PRE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = next[i];
        if (t + gridDim.x < tiles) load(next, t + gridDim.x);
      } else {
        load(w, t);
      }
      uint32_t m[8];
      tile_top(w, m);
      bool odd = false;             // an infinity or NaN somewhere in the tile
#pragma unroll
      for (int j = 0; j < 8; ++j) odd |= m[j] >= OPS_INF;
      odd = __syncthreads_or(odd);
      if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[8];
          w[i].values(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
            if (a < OPS_INF) m[j] = max(m[j], a);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
      if ((tid & 16) == 0) {
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          *reinterpret_cast<uint4*>(&part[warp][tc * 8 + j]) = make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
      }
      __syncthreads();
      if (tid < 128) {
        uint32_t a = part[0][tid];
#pragma unroll
        for (int k = 1; k < 8; ++k) a = max(a, part[k][tid]);
        if (MODE != T_COLS_T) {
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
          if ((tid & 31) == 0) part[0][tid] = a;      // read by this thread's own warp alone so far
        } else {
          uint32_t e;
          inv[tid] = ops_scale(a, &e);
          if (ct * 128 + tid < cols) o.s[(long long)(b * cols + ct * 128 + tid) * o.lds + rt] = (uint8_t)e;
        }
      }
      __syncthreads();
      float s0 = 1.f;
      if (MODE != T_COLS_T) {
        uint32_t e0;
        s0 = ops_scale(max(max(part[0][0], part[0][32]), max(part[0][64], part[0][96])), &e0);
        if (tid == 0) {
          if (MODE == T_BLOCK) o.s[(long long)(b * ((rows + 127) / 128) + rt) * o.lds + ct] = (uint8_t)e0;
          else o.s[(long long)(b * ((cols + 127) / 128) + ct) * o.lds + rt] = (uint8_t)e0;
        }
      }
      if (MODE == T_BLOCK) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[8];
          w[i].values(v);
          if (odd) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ops_finite(v[j]);
          }
          if (r0 + i < rows) ops_st_codes<VEC>(o.q + (long long)(b * rows + r0 + i) * o.ld, c0, cols, ops_codes8(v, s0), true);
        }
      } else {
        float sc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = MODE == T_COLS_T ? inv[tc * 8 + j] : s0;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          float v[4][8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[i + k].values(v[k]);
            if (odd) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[k][j] = ops_finite(v[k][j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            reinterpret_cast<uint32_t*>(tile)[((tc * 8 + j) * 16 + (tr ^ tc)) * 2 + i / 4] =
                ops_codes4(v[0][j], v[1][j], v[2][j], v[3][j], sc[j]);
        }
        __syncthreads();
        const int left = lim - rt * 128;     // codes of an output row in this tile
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = (tid >> 3) + 32 * i, k = (tid & 7) * 2;
          if (ct * 128 + c < cols) {
            const uint2 a = tile[c * 16 + (k ^ (c >> 3))], d = tile[c * 16 + ((k + 1) ^ (c >> 3))];
            uint8_t* p = o.q + (long long)(b * cols + ct * 128 + c) * o.ld + rt * 128;
            if (k * 8 + 16 <= left) {
              *reinterpret_cast<uint4*>(p + k * 8) = make_uint4(a.x, a.y, d.x, d.y);
            } else {
              ops_st_codes<0>(p, k * 8, left, a, false);
              ops_st_codes<0>(p, k * 8 + 8, left, d, false);
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// SwiGLU
// ---------------------------------------------------------------------------
// 1 / (1 + 2^(-g log2 e)) on the two approximate instructions (2 and 1 ulp): the
// product's rounding adds |g| 2^-24, far inside the 8-bit results' steps.  Below
// g = -87.3, where it is under 2^-126, it is 0.
__device__ __forceinline__ float sigmoid_f(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// Half a warp holds one block of g and the same block of u: act and, where
// asked for, g and u leave as codes in the same pass.  R rows per warp, loads first.
template <class T, int VEC, bool SAVE, int R>
__global__ void __launch_bounds__(256, SAVE ? 4 : 1) swiglu_k(const T* gu, long long ldgu, const int* n_rows, Mat8 act, Mat8 sv) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int F = act.cols, lim = ops_row_limit(n_rows, act.rows), nb = (F + 127) / 128;
  const int r0 = ((int)blockIdx.x * 8 + warp) * R;
  if (r0 >= lim) return;
  const bool v8 = (F & 7) == 0;
  for (int c = lane * 8 + 256 * (int)blockIdx.y; c - lane * 8 < F; c += 256 * (int)gridDim.y) {
    Raw8<T> g8[R], u8[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* p = gu + (long long)min(r0 + i, lim - 1) * ldgu;
      g8[i].template load<VEC>(p, c, F);
      u8[i].template load<VEC>(p + F, c, F);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const long long r = r0 + i;
      if (r >= lim) break;
      const bool first = (lane & 15) == 0 && c < F;
      float g[8], u[8], a[8];
      g8[i].values(g);
      u8[i].values(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = g[j] * sigmoid_f(g[j]) * u[j];
      uint32_t e;
      const uint2 q = ops_quantise(a, ops_max16(ops_top8(a)), &e);
      ops_st_codes<VEC>(act.q + r * act.ld, c, F, q, true);
      if (first) act.s[r * act.lds + (c >> 7)] = (uint8_t)e;
      if (SAVE) {
        uint32_t eg, eu;
        uint32_t tg = g8[i].top(), tu = u8[i].top();
        if (sizeof(T) == 2) {            // 16 bits each: one word goes round
          uint32_t t = (tg >> 16) | tu;
#pragma unroll
          for (int d = 8; d > 0; d >>= 1) t = ops_max_u16x2(t, __shfl_xor_sync(0xffffffffu, t, d));
          tg = t << 16;
          tu = t & 0xffff0000u;
        } else {
          tg = ops_max16(tg);
          tu = ops_max16(tu);
        }
        const uint2 qg = ops_quantise(g, tg, &eg), qu = ops_quantise(u, tu, &eu);
        ops_st_codes<VEC>(sv.q + r * sv.ld, c, F, qg, true);
        ops_st_codes<VEC>(sv.q + r * sv.ld + F, c, F, qu, v8);
        if (first) {
          sv.s[r * sv.lds + (c >> 7)] = (uint8_t)eg;
          sv.s[r * sv.lds + nb + (c >> 7)] = (uint8_t)eu;
        }
      }
    }
  }
}

template <class T, int VEC>
__global__ void __launch_bounds__(256) swiglu_bwd_k(const T* da, long long ldda, Mat8 sv, const int* n_rows, T* dgu,
                                                    long long lddgu, T* act, long long ldact) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int F = sv.cols / 2, lim = ops_row_limit(n_rows, sv.rows), nb = (F + 127) / 128;
  const long long r = (long long)blockIdx.x * 8 + warp;
  if (r >= lim) return;
  const bool v8 = (F & 7) == 0;
  for (int c = lane * 8 + 256 * (int)blockIdx.y; c < F; c += 256 * (int)gridDim.y) {
    float d[8], g[8], u[8], a[8];
    ops_ld8<VEC>(da + r * ldda, c, F, d);
    const uint2 qg = ops_ld_codes<VEC>(sv.q + r * sv.ld, c, F, true);
    const uint2 qu = ops_ld_codes<VEC>(sv.q + r * sv.ld + F, c, F, v8);
    const uint32_t eg = sv.s[r * sv.lds + (c >> 7)], eu = sv.s[r * sv.lds + nb + (c >> 7)];
    ops_values8(qg, ops_byte_scale(eg), g);
    ops_values8(qu, ops_byte_scale(eu), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid_f(g[j]), gs = g[j] * s, x = d[j];
      a[j] = gs * u[j];
      d[j] = x * u[j] * (s + gs * (1.f - s));
      u[j] = x * gs;
    }
    ops_st8<VEC>(dgu + r * lddgu, c, F, d);
    ops_st8<VEC>(dgu + r * lddgu + F, c, F, u);
    if (act) ops_st8<VEC>(act + r * ldact, c, F, a);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Rows per warp: one where that still leaves every SM fewer than 16 warps, so
// that small matrices spread; four otherwise, for loads in flight.
int rows_per_warp(int64_t rows, int64_t cols) { return rows * ((cols + 255) / 256) <= 152 * 16 ? 1 : 4; }
unsigned row_ctas(int64_t rows, int r) { return (unsigned)((rows + 8 * r - 1) / (8 * r)); }
unsigned col_ctas(int64_t cols, int per) {
  const int64_t n = (cols + per - 1) / per;
  return (unsigned)(n < 1024 ? n : 1024);
}

template <class T, int VEC>
int quant_rows_t(const void* x, int64_t ldx, const int* n_rows, const mt_mat8* o, cudaStream_t st) {
  const int parts = o->halves ? 2 : 1;
  const int64_t pc = o->cols / parts, chunks = (pc + 255) / 256 * parts;
  const int r = rows_per_warp(o->rows, chunks * 256);
  return ops_launch(r == 1 ? quant_rows_k<T, VEC, 1> : quant_rows_k<T, VEC, 4>,
                    dim3(row_ctas(o->rows, r), col_ctas(chunks, 1)), 256, 0, st, 1, (const T*)x, ldx, n_rows, mat8(o),
                    parts, pc);
}
template <class T, int VEC, int MODE>
int quant_tile_t(const void* x, int64_t ldx, const Src8& src, const int* n_rows, const mt_mat8* o, int64_t rows,
                 int64_t cols, cudaStream_t st) {
  const int64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
  const int64_t most = (152 * (sizeof(T) == 1 ? 3 : 2) + o->batch - 1) / o->batch;     // the CTAs that fit at one time
  const dim3 grid((unsigned)(tiles < most ? tiles : most), 1, (unsigned)o->batch);
  return ops_launch(quant_tile_k<T, VEC, MODE>, grid, 256, 0, st, 1, (const T*)x, ldx, src, n_rows, mat8(o), rows, cols);
}
template <class T, int VEC>
int dequant_t(const mt_mat8* a, const int* n_rows, void* out, int64_t ldo, cudaStream_t st) {
  const int parts = a->halves ? 2 : 1;
  const int64_t pc = a->cols / parts, chunks = (pc + 255) / 256 * parts;
  return ops_launch(dequant_k<T, VEC>, dim3(row_ctas(a->rows, 4), col_ctas(chunks, 1)), 256, 0, st, 1, mat8(a), n_rows,
                    parts, pc, (T*)out, ldo);
}
// With checkpoints two rows per warp share the loads' trip (52 -> 46 us at 65536 x
// 512, 64 registers); without, and backward, more warps do better (33 -> 30 and 64
// -> 54 us).
template <class T, int VEC>
int swiglu_t(const void* gu, int64_t ldgu, const int* n_rows, const mt_mat8* act, const mt_mat8* sv,
             cudaStream_t st) {
  const int r = !sv || rows_per_warp(act->rows, act->cols) == 1 ? 1 : 2;
  auto k = !sv ? swiglu_k<T, VEC, false, 1> : r == 1 ? swiglu_k<T, VEC, true, 1> : swiglu_k<T, VEC, true, 2>;
  return ops_launch(k, dim3(row_ctas(act->rows, r), col_ctas(act->cols, 256)), 256, 0, st, 1, (const T*)gu, ldgu,
                    n_rows, mat8(act), sv ? mat8(sv) : Mat8{});
}
template <class T, int VEC>
int swiglu_bwd_t(const void* da, int64_t ldda, const mt_mat8* sv, const int* n_rows, void* dgu, int64_t lddgu,
                 void* act, int64_t ldact, cudaStream_t st) {
  return ops_launch(swiglu_bwd_k<T, VEC>, dim3(row_ctas(sv->rows, 1), col_ctas(sv->cols / 2, 256)), 256, 0, st, 1,
                    (const T*)da, ldda, mat8(sv), n_rows, (T*)dgu, lddgu, (T*)act, ldact);
}

// Instantiations by element type and access mode (see ops_ld8); a second part of
// the columns has to start as well aligned as the row.
int part_vec(int vec, int dtype, int64_t part) {
  const int64_t b = part * ops_size(dtype);
  return ops_least(vec, b % (8 * ops_size(dtype)) == 0 ? 2 : b % 16 == 0 ? 1 : 0);
}
#define OPS_PICK(f, dtype, vec, ...)                                                                     \
  ((dtype) == MT_DT_FP32 ? ((vec) == 2 ? f<float, 2 __VA_ARGS__> : (vec) ? f<float, 1 __VA_ARGS__> : f<float, 0 __VA_ARGS__>) \
                         : ((vec) == 2 ? f<__nv_bfloat16, 2 __VA_ARGS__>                                 \
                            : (vec)    ? f<__nv_bfloat16, 1 __VA_ARGS__>                                 \
                                       : f<__nv_bfloat16, 0 __VA_ARGS__>))
#define OPS_COMMA ,

bool limit_ok(const int32_t* n_rows) { return !n_rows || ops_aligned(n_rows, 4); }

}  // namespace

extern "C" {

int32_t mt_quant8(const void* x, int32_t dtype, int64_t ldx, const int32_t* n_rows, const mt_mat8* out, void* stream) {
  if (!ops_mat8_ok(out) || !ops_dtype_ok(dtype) || !limit_ok(n_rows)) return MT_ERR_ARG;
  if (n_rows && (out->batch != 1 || out->block_rows != 1)) return MT_ERR_ARG;
  if (out->rows == 0) return MT_OK;
  if (!ops_mat_ok(x, dtype, ldx, out->cols)) return MT_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int vec = ops_vec(x, dtype, ldx);
  if (out->block_rows == 1) {
    mt_mat8 o = *out;            // stacked matrices are one tall one
    o.rows *= o.batch;
    const int64_t part = o.halves ? o.cols / 2 : o.cols;
    const int v = ops_mode(o.halves ? part_vec(vec, dtype, part) : vec, part, 256);
    return OPS_PICK(quant_rows_t, dtype, v)(x, ldx, n_rows, &o, st);
  } else {
    if (out->batch > 65535) return MT_ERR_UNSUPPORTED;
    const Src8 none{};
    const int v = ops_mode(vec, out->cols, 128);
    return OPS_PICK(quant_tile_t, dtype, v, OPS_COMMA T_BLOCK)(x, ldx, none, nullptr, out, out->rows, out->cols, st);
  }
}

int32_t mt_quant8_t(const void* x, int32_t dtype, int64_t ldx, const mt_mat8* x8, const int32_t* n_rows,
                    const mt_mat8* out, void* stream) {
  if (!ops_mat8_ok(out) || out->halves || !limit_ok(n_rows)) return MT_ERR_ARG;
  if (n_rows && out->batch != 1) return MT_ERR_ARG;
  if ((x != nullptr) == (x8 != nullptr) && out->rows) return MT_ERR_ARG;
  if (out->rows == 0) return MT_OK;
  if (out->batch > 65535) return MT_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t rows = out->cols, cols = out->rows;
  if (x8) {
    if (!ops_mat8_ok(x8) || x8->block_rows != 1 || x8->batch != 1 || x8->halves || out->batch != 1 || x8->rows != rows ||
        x8->cols != cols)
      return MT_ERR_ARG;
    const Src8 src{(const uint8_t*)x8->codes, (const uint8_t*)x8->scales, x8->ld, x8->lds};
    auto f = out->block_rows == 1 ? (cols % 128 ? quant_tile_t<uint8_t, 1, T_COLS_T> : quant_tile_t<uint8_t, 2, T_COLS_T>)
                                  : (cols % 128 ? quant_tile_t<uint8_t, 1, T_BLOCK_T> : quant_tile_t<uint8_t, 2, T_BLOCK_T>);
    return f(nullptr, 0, src, n_rows, out, rows, cols, st);
  }
  if (!ops_dtype_ok(dtype) || !ops_mat_ok(x, dtype, ldx, cols)) return MT_ERR_ARG;
  const int v = ops_mode(ops_vec(x, dtype, ldx), cols, 128);
  const Src8 none{};
  auto f = out->block_rows == 1 ? OPS_PICK(quant_tile_t, dtype, v, OPS_COMMA T_COLS_T)
                                : OPS_PICK(quant_tile_t, dtype, v, OPS_COMMA T_BLOCK_T);
  return f(x, ldx, none, n_rows, out, rows, cols, st);
}

int32_t mt_dequant8(const mt_mat8* a, const int32_t* n_rows, void* out, int32_t dtype, int64_t ldo, void* stream) {
  if (!ops_mat8_ok(a) || a->block_rows != 1 || a->batch != 1 || !ops_dtype_ok(dtype) || !limit_ok(n_rows))
    return MT_ERR_ARG;
  if (a->rows == 0) return MT_OK;
  if (!ops_mat_ok(out, dtype, ldo, a->cols)) return MT_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t part = a->halves ? a->cols / 2 : a->cols;
  const int vec = ops_vec(out, dtype, ldo), v = ops_mode(a->halves ? part_vec(vec, dtype, part) : vec, part, 256);
  return OPS_PICK(dequant_t, dtype, v)(a, n_rows, out, ldo, st);
}

int32_t mt_swiglu8(const void* gu, int32_t dtype, int64_t ldgu, const int32_t* n_rows, const mt_mat8* act,
                   const mt_mat8* saved, void* stream) {
  if (!ops_mat8_ok(act) || act->block_rows != 1 || act->batch != 1 || act->halves || !ops_dtype_ok(dtype) ||
      !limit_ok(n_rows))
    return MT_ERR_ARG;
  if (saved && (!ops_mat8_ok(saved) || saved->block_rows != 1 || saved->batch != 1 || !saved->halves ||
                saved->rows != act->rows || saved->cols != 2 * act->cols))
    return MT_ERR_ARG;
  if (act->rows == 0) return MT_OK;
  if (!ops_mat_ok(gu, dtype, ldgu, 2 * act->cols)) return MT_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int v = ops_mode(part_vec(ops_vec(gu, dtype, ldgu), dtype, act->cols), act->cols, 256);
  return OPS_PICK(swiglu_t, dtype, v)(gu, ldgu, n_rows, act, saved, st);
}

int32_t mt_swiglu8_bwd(const void* dact, int32_t dtype, int64_t ldda, const mt_mat8* saved, const int32_t* n_rows,
                       void* dgu, int64_t lddgu, void* act, int64_t ldact, void* stream) {
  if (!ops_mat8_ok(saved) || saved->block_rows != 1 || saved->batch != 1 || !saved->halves || !ops_dtype_ok(dtype) ||
      !limit_ok(n_rows))
    return MT_ERR_ARG;
  if (saved->rows == 0) return MT_OK;
  const int64_t F = saved->cols / 2;
  if (!ops_mat_ok(dact, dtype, ldda, F) || !ops_mat_ok(dgu, dtype, lddgu, 2 * F) ||
      (act && !ops_mat_ok(act, dtype, ldact, F)))
    return MT_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int vec = ops_least(ops_vec(dact, dtype, ldda), ops_least(ops_vec(dgu, dtype, lddgu), act ? ops_vec(act, dtype, ldact) : 2));
  const int v = ops_mode(part_vec(vec, dtype, F), F, 256);
  return OPS_PICK(swiglu_bwd_t, dtype, v)(dact, ldda, saved, n_rows, dgu, lddgu, act, ldact, st);
}

}  // extern "C"
