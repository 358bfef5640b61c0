// block_norm.cu - the joint between two blocks (mt_block_norm) and its gradients
// (mt_block_norm_bwd): norm after a block, gate, scaled residual sum, norm
// before the next block.
#include <math.h>
#include <string.h>

#include "ops8.cuh"

namespace {

#define BN_MAX_WIDTH 8192
#define BN_MAX_PARTS 160          // CTAs that leave partial column sums
#define BN_WARPS 16               // of a CTA of the backward pass
#define BN_SMEM (226 * 1024)      // its shared memory
#define BN_STAGES 2               // of its ring, at most (three: 83 against 80 us)

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
  float* ws;                      // [CTAs][sums][width], see bn_finish
  float *dafter, *dbefore;
  int accumulate;
  // elements from a group's row to its next
  long long hop_dh, hop_h, hop_dr, hop_y, hop_gate, hop_dx, hop_dy, hop_dgate;
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
// many warps as they have 1024 columns.  Memory bounds it: 45 to 50 us for 25 million
// elements (fp32 stream, bf16) in rows of 256 to 8192, 89 to 98 % of the copy rate, and 53
// in rows of 8000; a warp to 256 columns takes 102 us for rows of 256, 47 for 768 and 85
// for 8192.  Shorter rows leave lanes idle (128 columns 66 us, 64 124), rows by element
// take narrow loads and stores (1001: 86).
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
// two fp32 numbers in a register pair: one issue slot for both
typedef unsigned long long bn2;
__device__ __forceinline__ bn2 bn_pair(float x, float y) {
  bn2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void bn_split(bn2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ bn2 bn_mul(bn2 a, bn2 b) {
  bn2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ bn2 bn_fma(bn2 a, bn2 b, bn2 c) {
  bn2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float bn_both(bn2 v) {
  float x, y;
  bn_split(v, x, y);
  return x + y;
}
__device__ __forceinline__ void bn_pairs(const float* v, bn2* p) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = bn_pair(v[2 * e], v[2 * e + 1]);
}
template <class T>
__device__ __forceinline__ void bn_pairs(const Raw8<T>& r, bn2* p) {
  float v[8];
  r.values(v);
  bn_pairs(v, p);
}
template <int VEC, class T>
__device__ __forceinline__ void bn_store(T* p, int c, int n, const bn2* v) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) bn_split(v[e], x[2 * e], x[2 * e + 1]);
  bn_store<VEC>(p, c, n, x);
}

// Sums over a group of `warps` warps (named barrier `bar`), for every lane.  red:
// two buffers of four words a warp, taken in turn: whoever writes one again has
// passed the other's barrier, and with it every warp's reads of this one.
struct Group {
  float* red;
  int warps, w, lane, bar, turn;
  __device__ __forceinline__ float* mine() const { return red + (turn * warps + w) * 4; }
  __device__ __forceinline__ const float* meet() {
    const float* r = red + turn * warps * 4;
    turn ^= 1;
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * warps) : "memory");
    return r;
  }
  __device__ __forceinline__ float sum(float a) {
    a = bn_sum(a);
    if (lane == 0) *mine() = a;
    const float* r = meet();
    a = 0.f;
    for (int i = 0; i < warps; ++i) a += r[i * 4];
    return a;
  }
  // three at once, in 6 shuffles instead of 15: after two exchanges a lane has one of
  // them only - first, second, third, second by eights of lanes
  __device__ __forceinline__ void sum(float& a, float& b, float& c) {
    const bool h16 = lane & 16, h8 = lane & 8;
    float x = (h16 ? c : a) + __shfl_xor_sync(0xffffffffu, h16 ? a : c, 16);
    const float y = b + __shfl_xor_sync(0xffffffffu, b, 16);
    x = (h8 ? y : x) + __shfl_xor_sync(0xffffffffu, h8 ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((lane & 7) == 0) mine()[lane >> 3] = x;
    const float* r = meet();
    a = b = c = 0.f;
    for (int i = 0; i < warps; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(r + i * 4);
      a += v.x;
      b += v.y;
      c += v.z;
    }
  }
};

// Rows of whole eights go through a ring in shared memory that a warp has to itself,
// copied there 16 bytes at a time while it works on the rows before: no registers
// hold them.  An array's eights of a warp take 32 pieces of 16 bytes (bf16; a lane
// copies its own) or 64 (fp32; lane l copies pieces l and 32 + l, so that a copy
// instruction takes whole sectors: a lane's own two would ask L2 for every sector
// twice, 104 against 88 us at 32,768 x 768).  fp32 piece p lies at p ^ (p >> 3 & 1):
// neither the copies nor the lanes' reads of pieces 2 l and 2 l + 1 meet a bank twice.
template <class T>
struct Piece {
  static constexpr int N = (int)sizeof(T) / 2;          // pieces of eight elements
  // a lane's first copy: its column within the warp's 256, its place in the array's part
  __device__ __forceinline__ static int column(int lane) { return N == 2 ? lane * 4 : lane * 8; }
  __device__ __forceinline__ static uint32_t place(int wid, int lane) {
    return (uint32_t)(N == 2 ? wid * 64 + (lane ^ (lane >> 3 & 1)) : wid * 32 + lane) * 16;
  }
};
__device__ __forceinline__ void bn_copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// columns c (and c + 128) of the row at p, as far as it has them
template <class T>
__device__ __forceinline__ void bn_copy(uint32_t to, const T* p, int c, int n) {
  if (c < n) bn_copy16(to, p);
  if (Piece<T>::N == 2 && c + 128 < n) bn_copy16(to + 512, p + 128);
}
// eight elements of this lane as four pairs
__device__ __forceinline__ void bn_take(const __nv_bfloat16*, uint32_t at, int wid, int lane, bn2* p) {
  Raw8<__nv_bfloat16> v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.u.x), "=r"(v.u.y), "=r"(v.u.z), "=r"(v.u.w)
               : "r"(at + (wid * 32 + lane) * 16)
               : "memory");
  bn_pairs(v, p);
}
__device__ __forceinline__ void bn_take(const float*, uint32_t at, int wid, int lane, bn2* p) {
  const uint32_t a = at + (uint32_t)(wid * 64 + (2 * lane ^ (lane >> 2 & 1))) * 16;
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(p[0]), "=l"(p[1]) : "r"(a) : "memory");
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(p[2]), "=l"(p[3]) : "r"(a ^ 16) : "memory");
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
// What a sum over all rows gives: the first (of two, or the only one, with `before`) is
// dbefore, the other q.  The factors and what is added to are read before any of U
// columns is written.
template <int U>
__device__ __forceinline__ void bn_finish(const Bwd& f, const int (&k)[U], const int (&c)[U], const float (&v)[U]) {
  const bool channel = f.j.gate_kind == MT_GATE_CHANNEL;
  const float* gate = (const float*)f.j.gate;
  float* dgate = (float*)f.dgate;
  float ga[U], af[U], o1[U], o2[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    ga[u] = af[u] = 1.f;
    o1[u] = o2[u] = 0.f;
    if (c[u] >= f.j.width) continue;
    if (k[u] == 0 && f.j.before) {
      if (f.accumulate) o1[u] = f.dbefore[c[u]];
      continue;
    }
    if (channel && f.j.after) ga[u] = gate[c[u]], af[u] = f.j.after[c[u]];
    if (f.accumulate && f.j.after) o1[u] = f.dafter[c[u]];
    if (f.accumulate && channel) o2[u] = dgate[c[u]];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (c[u] >= f.j.width) continue;
    if (k[u] == 0 && f.j.before) {
      f.dbefore[c[u]] = o1[u] + v[u];
      continue;
    }
    // rounded before it is added: a gradient added is the gradient alone, added
    if (f.j.after) f.dafter[c[u]] = o1[u] + __fmul_rn(v[u], ga[u]);
    if (channel) dgate[c[u]] = o2[u] + __fmul_rn(v[u], af[u]);
  }
}

// bytes of the groups' sums, below the ring, which starts on a line of all banks (80.9
// us off one where 76.1 on one)
__host__ __device__ constexpr int bn_red(int warps) { return (warps * 32 + 127) / 128 * 128; }

// Persistent CTAs of G groups; a group of W warps takes a row, a lane 8 C fixed
// columns of it, so the gains and the column sums stay in registers from row to
// row.  With rh = 1 / rms(h), u = dr * before, t the token's gate (1 without one):
//   G = dh + rh u - h rh^3 mean(u h)              dx = a G, dbefore += dr h rh
//   x = b G (full gate: times the gate), p = x * after * channel gate
//   s = sum(p y)                                  dgate of a token = s ry
//   dy = t (p ry - y ry^3 s / width)              q += t x y ry
// and after the last row dafter = q * channel gate, a channel gate's gradient q *
// after: one sum for both.  A full gate's gradient is b G y ry after.  Two sums over
// the row: (h^2, u h, y^2) and s.  VEC: the next stages - 1 rows are on their way in
// the ring, and what a phase needs of a row is read from there again.  Otherwise the
// next row is on its way in registers (C 1).
// 32,768 x 768 (fp32 stream, bf16, a channel gate), us with the column sums: 76, 88 %
// of the copy rate; rows in registers 109, two rows at once 87 to 90, a warp to a row
// of three chunks 83 and more, 20 warps 86, 8 warps 138.  As many elements in rows of
// other widths: 64 222 and 128 117 (idle lanes), 2048 84, 2304 106 (nine of sixteen warps
// run), 4096 97 (one row at a time, its sums over all warps), 5120 118 and 8000 108 (and
// registers spilled), by element 1001 135 (narrow loads, and in fp32 registers spilled).
template <class S, class T, int VEC, int C, bool ALL, int WARPS = BN_WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) block_norm_bwd_k(Bwd f, int W, int G, int stages, int pieces) {
  ops_begin();
  extern __shared__ __align__(128) float sh[];
  constexpr int NS = Piece<S>::N, NT = Piece<T>::N;
  const Joint& j = f.j;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = wid / W, w = wid - g * W, n = j.width;
  Group grp = {sh + g * W * 8, W, w, lane, 1 + g, 0};
  const int lim = ops_row_limit(j.n_rows, j.rows), step = (int)gridDim.x * G;
  const float mean = 1.f / (float)n;
  // ALL: every part but a gate is there, known when this was compiled
  const bool has_b = ALL || j.before, has_a = ALL || j.after, has_y = ALL || f.y, has_dh = ALL || f.dh;
  const bool channel = j.gate_kind == MT_GATE_CHANNEL, token = j.gate_kind == MT_GATE_TOKEN,
             full = j.gate_kind == MT_GATE_FULL;
  // gains of a lane's columns: kept, but by element and C 2 fetched where they are used
  constexpr bool KEEP = VEC || C == 1;
  bn2 kb[C][4], kw[C][4], sb[C][4], sq[C][4];
  auto before = [&](int i) {
    float v[8];
    bn_vec<VEC>(j.before, bn_col<VEC>(w + i * W, lane), n, v);
    bn_pairs(v, kb[i]);
  };
  auto behind = [&](int i) {
    const int c = bn_col<VEC>(w + i * W, lane);
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
    if (has_a) bn_vec<VEC>(j.after, c, n, v);
    if (channel) {
      bn_vec<VEC>((const float*)j.gate, c, n, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= u[e];
    }
    bn_pairs(v, kw[i]);
  };
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sb[i][e] = sq[i][e] = 0;
    if (KEEP && has_b) before(i);
    if (KEEP && has_y) behind(i);
  }
  BwdRow<S, T> cur[C];
  long long row = (long long)blockIdx.x * G + g;
  const uint32_t hop = blockDim.x * 16, unit = hop * pieces, slot = unit * C;   // a piece; a lane's eight; a stage
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sh) + bn_red(G * W);
  uint32_t put = 0, get = 0;
  // where the next row to send lies, for a lane's first copies; a row's hop is a
  // parameter of its own
  const int cs = w * 256 + Piece<S>::column(lane), ct = w * 256 + Piece<T>::column(lane);
  const uint32_t at_s = Piece<S>::place(wid, lane), at_t = Piece<T>::place(wid, lane);
  int ahead = (int)row;
  const S *p_dh = nullptr, *p_h = nullptr;
  const T *p_dr = nullptr, *p_y = nullptr, *p_gate = nullptr;
  if (has_dh) p_dh = (const S*)f.dh + row * f.lddh + cs;
  if (has_b) p_h = (const S*)f.h + row * f.ldh + cs;
  if (has_b) p_dr = (const T*)f.dr + row * f.lddr + ct;
  if (has_y) p_y = (const T*)f.y + row * f.ldy + ct;
  if (full) p_gate = (const T*)j.gate + row * j.ldgate + ct;
  auto send = [&]() {
    if (ahead < lim) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const uint32_t to = ring + put + i * unit;
        const int c = i * W * 256;
        if (has_dh) bn_copy(to + at_s, p_dh + c, cs + c, n);
        if (has_b) {
          bn_copy(to + NS * hop + at_s, p_h + c, cs + c, n);
          bn_copy(to + 2 * NS * hop + at_t, p_dr + c, ct + c, n);
        }
        if (has_y) bn_copy(to + (2 * NS + NT) * hop + at_t, p_y + c, ct + c, n);
        if (full) bn_copy(to + (2 * NS + 2 * NT) * hop + at_t, p_gate + c, ct + c, n);
      }
      ahead += step;
      p_dh += f.hop_dh;
      p_h += f.hop_h;
      p_dr += f.hop_dr;
      p_y += f.hop_y;
      if (full) p_gate += f.hop_gate;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + slot == slot * stages ? 0 : put + slot;
  };
  // a row's inputs as pairs, of chunk i
  auto in_h = [&](int i, bn2* p) {
    if constexpr (VEC) bn_take((const S*)nullptr, ring + get + i * unit + NS * hop, wid, lane, p);
    else bn_pairs(cur[i].h, p);
  };
  auto in_dh = [&](int i, bn2* p) {
    if constexpr (VEC) bn_take((const S*)nullptr, ring + get + i * unit, wid, lane, p);
    else bn_pairs(cur[i].dh, p);
  };
  auto in_dr = [&](int i, bn2* p) {
    if constexpr (VEC) bn_take((const T*)nullptr, ring + get + i * unit + 2 * NS * hop, wid, lane, p);
    else bn_pairs(cur[i].dr, p);
  };
  auto in_y = [&](int i, bn2* p) {
    if constexpr (VEC) bn_take((const T*)nullptr, ring + get + i * unit + (2 * NS + NT) * hop, wid, lane, p);
    else bn_pairs(cur[i].y, p);
  };
  auto in_gate = [&](int i, bn2* p) {
    if constexpr (VEC) bn_take((const T*)nullptr, ring + get + i * unit + (2 * NS + 2 * NT) * hop, wid, lane, p);
    else bn_pairs(cur[i].gate, p);
  };
  if constexpr (VEC) {
    // columns behind the row stay zeros in every stage
    if (n < 256 * C * W) {
      for (uint32_t at = threadIdx.x * 16; at < slot * stages; at += hop)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + at), "r"(0) : "memory");
      __syncthreads();
    }
    for (int k = 0; k < stages - 1; ++k) send();
  } else if (C == 1 && row < lim) {
    bn_row<VEC>(cur[0], f, row, bn_col<VEC>(w, lane));
  }
  S* o_dx = (S*)f.dx + row * f.lddx;
  T *o_dy = nullptr, *o_dgate = nullptr;
  if (has_y) o_dy = (T*)f.dy + row * f.lddy;
  if (full) o_dgate = (T*)f.dgate + row * f.lddgate;
  const bn2 a2 = bn_pair(j.a, j.a), b2 = bn_pair(j.b, j.b);
  for (; row < lim; row += step) {
    BwdRow<S, T> next = cur[0];
    if constexpr (VEC) {
      if (row != (long long)blockIdx.x * G + g) __syncwarp();    // the stage that this fills has been read
      send();
      // all but the newest stages - 1 copies have landed
      if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
      else asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();                                             // by every lane
    } else if constexpr (C > 1) {
#pragma unroll
      for (int i = 0; i < C; ++i) bn_row<VEC>(cur[i], f, row, bn_col<VEC>(w + i * W, lane));
    } else if (row + step < lim) {
      bn_row<VEC>(next, f, row + step, bn_col<VEC>(w, lane));
    }
    const float tg = token ? ((const float*)j.gate)[row * j.ldgate] : 1.f;
    bn2 hh = 0, uh = 0, yy = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      bn2 h[4], v[4];
      if (has_b) {
        if (!KEEP) before(i);
        in_h(i, h);
        in_dr(i, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hh = bn_fma(h[e], h[e], hh);
          uh = bn_fma(bn_mul(v[e], kb[i][e]), h[e], uh);
        }
      }
      if (has_a) {
        in_y(i, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) yy = bn_fma(v[e], v[e], yy);
      }
    }
    float s0 = bn_both(hh), s1 = bn_both(uh), s2 = bn_both(yy);
    grp.sum(s0, s1, s2);
    // rh^3 alone may be beyond fp32 for a small eps
    const float rh = rsqrtf(fmaf(s0, mean, j.eps)), qh = -(rh * (rh * (rh * (s1 * mean))));
    const float ry = has_a ? rsqrtf(fmaf(s2, mean, j.eps)) : 1.f, rt = ry * tg;
    const bn2 rh2 = bn_pair(rh, rh), qh2 = bn_pair(qh, qh), rt2 = bn_pair(rt, rt);
    bn2 gr[C][4], py = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = bn_col<VEC>(w + i * W, lane);
      bn2 h[4], v[4], o[4], (&x)[4] = gr[i];
      if (has_dh) {
        in_dh(i, x);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = 0;
      }
      if (has_b) {
        if (!KEEP) before(i);
        in_h(i, h);
        in_dr(i, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bn2 t = bn_mul(v[e], rh2);
          sb[i][e] = bn_fma(t, h[e], sb[i][e]);
          x[e] = bn_fma(t, kb[i][e], bn_fma(h[e], qh2, x[e]));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = bn_mul(a2, x[e]);
      bn_store<VEC>(o_dx, c, n, o);
      if (!has_y) continue;
      if (!KEEP) behind(i);
      in_y(i, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = bn_mul(b2, x[e]);
      if (full) {
        in_gate(i, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = bn_mul(bn_mul(x[e], kw[i][e]), bn_mul(v[e], rt2));
          x[e] = bn_mul(x[e], h[e]);
        }
        bn_store<VEC>(o_dgate, c, n, o);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sq[i][e] = bn_fma(x[e], bn_mul(v[e], rt2), sq[i][e]);
        x[e] = bn_mul(x[e], kw[i][e]);
        py = bn_fma(x[e], v[e], py);
      }
    }
    o_dx += f.hop_dx;
    if (full) o_dgate += f.hop_dgate;
    if (has_y) {
      float s = 0.f;
      if (has_a || token) s = grp.sum(bn_both(py));
      if (token && w == 0 && lane == 0) ((float*)f.dgate)[row * f.lddgate] = s * ry;
      const float qy = has_a ? -(rt * (ry * (ry * (s * mean)))) : 0.f;
      const bn2 qy2 = bn_pair(qy, qy);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        bn2 v[4];
        in_y(i, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bn_fma(gr[i][e], rt2, bn_mul(v[e], qy2));
        bn_store<VEC>(o_dy, bn_col<VEC>(w + i * W, lane), n, v);
      }
      o_dy += f.hop_dy;
    }
    if (VEC) get = get + slot == slot * stages ? 0 : get + slot;
    if (!VEC && C == 1) cur[0] = next;
  }
  // the groups' column sums side by side, then joined in the groups' order
  const int nb = has_b ? 1 : 0, nq = has_a || channel ? 1 : 0, ns = nb + nq;
  if (!ns) return;
  float* to = sh + (long long)g * ns * n;
  __syncthreads();                          // the rows' use of shared memory
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = bn_col<VEC>(w + i * W, lane);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 0 ? !nb : !nq) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) bn_split(k == 0 ? sb[i][e] : sq[i][e], v[2 * e], v[2 * e + 1]);
      float* p = to + (long long)(k ? nb : 0) * n;
      if constexpr (VEC) {
        if (c < n) {
          *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + 32 * e < n) p[c + 32 * e] = v[e];
      }
    }
  }
  __syncthreads();
  constexpr int U = 4;
  for (int c0 = threadIdx.x; c0 < ns * n; c0 += U * blockDim.x) {
    int k[U], c[U];
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c0 + u * (int)blockDim.x;
      k[u] = at >= n;
      c[u] = at < ns * n ? at - k[u] * n : n;
      v[u] = 0.f;
      for (int i = 0; i < G && c[u] < n; ++i) v[u] += sh[i * ns * n + at];
      if (gridDim.x > 1 && c[u] < n) f.ws[(long long)blockIdx.x * ns * n + at] = v[u];
    }
    if (gridDim.x == 1) bn_finish(f, k, c, v);
  }
}

// Sums of the CTAs' parts: eight warps take every eighth part of 32 columns, joined
// in order, with every load of a warp on its way at once (eight at a time: 5 us more),
// from L2, where other SMs left them.
// About 3 us behind the rows' kernel, of which its launch and one trip to L2 are most.
__global__ void __launch_bounds__(256) column_sums_k(Bwd f, int parts, int sums) {
  ops_begin();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, k = blockIdx.y, n = f.j.width;
  const float* at = f.ws + (long long)k * n + c;
  float v = 0.f;
  constexpr int U = 20;                       // all in flight: 152 parts by eight warps
  for (int p0 = w; p0 < parts && c < n; p0 += 8 * U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = p0 + 8 * u < parts ? __ldcg(at + (long long)(p0 + 8 * u) * sums * n) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) v += x[u];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w || c >= n) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += red[i][lane];
  const int ks[1] = {k}, cs[1] = {c};
  const float vs[1] = {v};
  bn_finish(f, ks, cs, vs);
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

// Warps of a row in the backward pass: one to 256 columns up to 4096, to 512 beyond.
int bn_width(int64_t width) {
  const int chunks = (int)((width + 255) / 256), C = chunks <= BN_WARPS ? 1 : 2;
  return (chunks + C - 1) / C;
}
// A few rows stay in one CTA, which leaves no parts: two rounds of its groups cost less
// than their sums (8 rows of 768: 6.0 against 6.4 us and a launch of the host's; three
// rounds: 7.3 against 6.4).
bool bn_alone(int64_t rows, int64_t width) { return rows <= 2 * (BN_WARPS / bn_width(width)); }

template <class S, class T, int VEC>
int bwd_t(Bwd f, int dev, int sms, int* parts, cudaStream_t st) {
  const int W = bn_width(f.j.width), C = W * 256 < f.j.width ? 2 : 1;
  const int pieces = 2 * Piece<S>::N + (f.j.gate_kind == MT_GATE_FULL ? 3 : 2) * Piece<T>::N;
  // rows are spread over the CTAs before any takes two at once
  const int most = ops_least(sms, BN_MAX_PARTS), room = W == 1 ? BN_WARPS - 1 : BN_WARPS / W;
  const bool alone = bn_alone(f.j.rows, f.j.width);
  const int G = alone ? room : ops_least(room, (f.j.rows + most - 1) / most);
  *parts = alone ? 1 : ops_least((f.j.rows + G - 1) / G, most);
  const size_t red = bn_red(G * W), stage = VEC ? (size_t)C * pieces * 512 * W * G : 0;
  int stages = BN_STAGES;
  while (stages > 1 && red + stages * stage > BN_SMEM) --stages;
  size_t smem = red + stages * stage, sums = (size_t)G * 2 * f.j.width * 4;
  if (smem < sums) smem = sums;
  const long long step = (long long)*parts * G;
  f.hop_dh = step * f.lddh, f.hop_h = step * f.ldh, f.hop_dr = step * f.lddr, f.hop_y = step * f.ldy;
  f.hop_gate = step * f.j.ldgate, f.hop_dx = step * f.lddx, f.hop_dy = step * f.lddy, f.hop_dgate = step * f.lddgate;
  auto k = C == 2 ? block_norm_bwd_k<S, T, VEC, 2, false> : block_norm_bwd_k<S, T, VEC, 1, false>;
  // compiled for a warp less it spills nothing: 75.8 against 80.0 us for 32,768 x 768
  // (five groups of three warps in both)
  if constexpr (VEC) {
    if (C == 1 && f.j.before && f.j.after && f.y && f.dh)
      k = W * G < BN_WARPS ? block_norm_bwd_k<S, T, VEC, 1, true, BN_WARPS - 1> : block_norm_bwd_k<S, T, VEC, 1, true>;
  }
  return ops_launch_wide(k, dev, BN_SMEM, (unsigned)*parts, 32u * W * G, smem, st, f, W, G, stages, pieces);
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
  if (bn_alone(rows, width)) return 0;
  return ((rows < BN_MAX_PARTS ? rows : BN_MAX_PARTS) * 2 * width * 4 + 15) / 16 * 16;
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
  const int sums = (dbefore ? 1 : 0) + (dafter || channel ? 1 : 0);
  const int64_t need = sums ? mt_block_norm_ws_bytes(j->rows, j->width) : 0;
  if (need && (!ws || !ops_aligned(ws, 16))) return MT_ERR_ARG;
  if (ws_bytes < need) return MT_ERR_ARENA_SMALL;
  cudaStream_t s = (cudaStream_t)stream;
  int parts = 0;
  const Bwd f = {joint(j), dr ? h : nullptr, y, dr, dh, dx, dy, dgate, ldh, ldy, lddr, lddh, lddx, lddy, lddgate, (float*)ws,
                 dafter, dbefore, accumulate};
  if (j->rows) {
    int dev, sms;
    if (!ops_device(&dev, &sms)) return MT_ERR_CUDA;
    const bool vec = joint_vec(j) && mat_vec(f.h, j->stream_dtype, ldh) && mat_vec(y, j->dtype, ldy) &&
                     mat_vec(dr, j->dtype, lddr) && mat_vec(dh, j->stream_dtype, lddh) &&
                     mat_vec(dx, j->stream_dtype, lddx) && mat_vec(dy, j->dtype, lddy) &&
                     (j->gate_kind != MT_GATE_FULL || mat_vec(dgate, j->dtype, lddgate));
    auto k = j->stream_dtype == MT_DT_BF16 ? (vec ? bwd_t<__nv_bfloat16, __nv_bfloat16, 1> : bwd_t<__nv_bfloat16, __nv_bfloat16, 0>)
             : j->dtype == MT_DT_BF16      ? (vec ? bwd_t<float, __nv_bfloat16, 1> : bwd_t<float, __nv_bfloat16, 0>)
                                           : (vec ? bwd_t<float, float, 1> : bwd_t<float, float, 0>);
    const int rc = k(f, dev, sms, &parts, s);
    if (rc || parts == 1) return rc;
  }
  if (!sums) return MT_OK;
  return ops_launch(column_sums_k, dim3((unsigned)((j->width + 31) / 32), (unsigned)sums), 256, 0, s, 1, f, parts, sums);
}

}  // extern "C"
