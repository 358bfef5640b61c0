// route_ops.cu - tokens sorted by expert and back (mt_route_order,
// mt_dispatch, mt_dispatch8, mt_combine, mt_combine_bwd).
#include "ops8.cuh"

namespace {

constexpr int RO_E = MT_MAX_EXPERTS;
constexpr int RO_SMALL = 4096;        // assignments that one CTA sorts alone,
constexpr int RO_CLUSTER = 1 << 16;   // that a cluster of sixteen sorts (65536: 6.3 us, a grid 7.5; 131072: 17 to 21, 15 to 17),
constexpr int RO_CTAS = 16;
constexpr int RO_CHUNK = 2048;        // and per CTA of a grid otherwise, or more:
constexpr int RO_GRID = 1024;         // its CTAs each add up the counts of all

// Expert of an assignment, -1 for none; counts indices out of range.
__device__ __forceinline__ int ro_expert(int e, int E, int* status) {
  if (e >= 0 && e < E) return e;
  if (e != -1 && atomicCAS(status, 0, (int)MT_ERR_DEVICE_BOUNDS) == 0) status[1] = 3;
  return -1;
}

// offs[0..E] of the padded segments, from the counts in cnt (first warp).
__device__ __forceinline__ void ro_offsets(const int* cnt, int E, int* offs) {
  const int l = threadIdx.x;
  if (l < 32) {
    const int c0 = 2 * l < E ? (cnt[2 * l] + 127) & ~127 : 0, c1 = 2 * l + 1 < E ? (cnt[2 * l + 1] + 127) & ~127 : 0;
    int s = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (l >= o) s += t;
    }
    if (l == 0) offs[0] = 0;
    if (2 * l < E) offs[2 * l + 1] = s - c1;
    if (2 * l + 1 < E) offs[2 * l + 2] = s;
  }
}

// Assignments a, a + 32, a + 64, a + 96; -1 from w1 on.
__device__ __forceinline__ void ro_load(const int* idx, long long a, long long w1, int* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = a + 32 * j < w1 ? idx[a + 32 * j] : -1;
}

// Lanes of the warp whose assignment names the same expert.
__device__ __forceinline__ unsigned ro_peers(int e) { return __match_any_sync(0xffffffffu, e); }

// Counting sort of assignments [a0, a1) by a CTA of NW warps, each warp taking
// `span` consecutive ones (a multiple of 32): wh[warp][e] counts, then holds the
// next row of expert e for the warp, so rows ascend with the assignment.  Chunks
// of a grid may be long: two reads of idx, the second from cache.
template <int NW>
struct RoSmem {
  int wh[NW][RO_E];
  int cnt[RO_E], before[RO_E], offs[RO_E + 1];
};

template <int NW>
__device__ __forceinline__ void ro_count(RoSmem<NW>& s, const int* idx, long long w0, long long w1, int E, int* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = lane; e < RO_E; e += 32) s.wh[warp][e] = 0;
  __syncwarp();
  for (long long a0 = w0; a0 < w1; a0 += 128) {
    int v[4];                            // four loads in flight
    ro_load(idx, a0 + lane, w1, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = ro_expert(v[j], E, status);
      const unsigned peers = ro_peers(e);
      if (e >= 0 && lane == __ffs(peers) - 1) s.wh[warp][e] += __popc(peers);
      __syncwarp();
    }
  }
}
template <int NW>
__device__ __forceinline__ void ro_place(RoSmem<NW>& s, const int* idx, long long w0, long long w1, int E, int* status,
                                         int* perm, int* row) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (long long a0 = w0; a0 < w1; a0 += 128) {
    int v[4];
    ro_load(idx, a0 + lane, w1, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long a = a0 + 32 * j + lane;
      const int e = ro_expert(v[j], E, status);
      const unsigned peers = ro_peers(e);
      int r = -1;
      if (e >= 0) {
        r = s.wh[warp][e] + __popc(peers & ((1u << lane) - 1u));
        perm[r] = (int)a;
      }
      if (a < w1) row[a] = r;
      __syncwarp();
      if (e >= 0 && lane == __ffs(peers) - 1) s.wh[warp][e] += __popc(peers);
      __syncwarp();
    }
  }
}
// -1 at the rows no assignment takes, spread over `nt` threads
__device__ __forceinline__ void ro_pads(const int* cnt, const int* offs, int E, long long rows, int* perm, long long t,
                                        long long nt) {
  for (long long i = t; i < (long long)E * 128; i += nt) {
    const int e = (int)(i >> 7);
    const int r = offs[e] + cnt[e] + (int)(i & 127);
    if (r < offs[e + 1]) perm[r] = -1;
  }
  for (long long r = offs[E] + t; r < rows; r += nt) perm[r] = -1;
}

__device__ __forceinline__ void ro_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void ro_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ int ro_remote(const int* p, int cta) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(cta));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Up to RO_SMALL assignments one CTA, up to RO_CLUSTER a cluster of sixteen whose
// CTAs read one another's counts in shared memory: one launch.  A lane keeps its
// choices and their places among the warp's equal ones in registers: idx is read
// once, all loads in flight, and the counts grow one time (65536 assignments 6.3
// us, 7.5 with a counting and a placing pass; 1024: 2.8 and 4.2).  Bound by
// latency: the choices' trip, the barriers, the serial counts of a warp.
template <int NC>
__global__ void __launch_bounds__(1024) ro_sort(const int* idx, int n, int E, long long rows, int* offs, int* perm,
                                                int* row, int* status) {
  ops_begin();
  constexpr int PER = (NC > 1 ? RO_CLUSTER : RO_SMALL) / (NC * 1024);   // choices of a lane, at most
  __shared__ RoSmem<32> s;
  __shared__ int start[RO_E];            // first row of this CTA's part of each segment
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int span = ((n + 32 * NC - 1) / (32 * NC) + 31) & ~31;
  const int w0 = min((cta * 32 + warp) * span, n), w1 = min(w0 + span, n);
  int mine[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) mine[j] = w0 + 32 * j + lane < w1 ? idx[w0 + 32 * j + lane] : -1;
  for (int e = lane; e < RO_E; e += 32) s.wh[warp][e] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (32 * j >= span) break;
    const int e = ro_expert(mine[j], E, status);
    const unsigned peers = ro_peers(e);
    int c = 0;
    if (e >= 0) c = s.wh[warp][e];
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) s.wh[warp][e] = c + __popc(peers);
    __syncwarp();
    mine[j] = e < 0 ? -1 : (c + __popc(peers & ((1u << lane) - 1u))) * RO_E + e;
  }
  __syncthreads();
  if (tid < RO_E) {
    int c = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const int t = s.wh[w][tid];
      s.wh[w][tid] = c;
      c += t;
    }
    s.before[tid] = c;                   // of this CTA, for the cluster
  }
  int base = 0;
  if (NC > 1) {
    ro_cluster_arrive();
    ro_cluster_wait();
    if (tid < RO_E) {
      int all = 0;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int t = ro_remote(&s.before[tid], c);
        if (c < cta) base += t;
        all += t;
      }
      s.cnt[tid] = all;
    }
    __syncwarp();
    ro_cluster_arrive();                 // the counts have been read
  } else if (tid < RO_E) {
    s.cnt[tid] = s.before[tid];
  }
  __syncthreads();
  ro_offsets(s.cnt, E, s.offs);
  __syncthreads();
  if (cta == 0 && tid <= E) offs[tid] = s.offs[tid];
  if (tid < E) start[tid] = s.offs[tid] + base;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int a = w0 + 32 * j + lane;
    if (a < w1) {
      const int e = mine[j] & (RO_E - 1);
      int r = -1;
      if (mine[j] >= 0) {
        r = start[e] + s.wh[warp][e] + mine[j] / RO_E;
        perm[r] = a;
      }
      row[a] = r;
    }
  }
  ro_pads(s.cnt, s.offs, E, rows, perm, cta * 1024 + tid, NC * 1024);
  if (NC > 1) ro_cluster_wait();         // no CTA's shared memory goes while another may read it
}

// Many: every CTA counts its chunk, then every CTA sums the counts before its
// own and places it.
__global__ void __launch_bounds__(256) ro_hist(const int* idx, long long n, int chunk, int E, int* hist, int* status) {
  ops_begin();
  __shared__ RoSmem<8> s;
  const long long a0 = (long long)blockIdx.x * chunk + (threadIdx.x >> 5) * (chunk / 8);
  const long long a1 = a0 + chunk / 8 < n ? a0 + chunk / 8 : n;
  ro_count(s, idx, a0, a1, E, status);
  __syncthreads();
  if (threadIdx.x < RO_E) {
    int c = 0;
    for (int w = 0; w < 8; ++w) c += s.wh[w][threadIdx.x];
    hist[(long long)blockIdx.x * RO_E + threadIdx.x] = c;
  }
}
__global__ void __launch_bounds__(256) ro_scatter(const int* idx, long long n, int chunk, int E, long long rows, const int* hist,
                                                  int* offs, int* perm, int* row, int* status) {
  ops_begin();
  __shared__ RoSmem<8> s;
  // counts come four experts per load: a thread adds up every sixteenth CTA's
  __shared__ __align__(16) int part[2][16][RO_E];
  const int tid = threadIdx.x, e = (tid & 15) * 4, p = tid >> 4;
  const long long a0 = (long long)blockIdx.x * chunk + (tid >> 5) * (chunk / 8);
  const long long a1 = a0 + chunk / 8 < n ? a0 + chunk / 8 : n;
  int4 all = make_int4(0, 0, 0, 0), mine = all;
  for (int c0 = p; c0 < (int)gridDim.x; c0 += 128) {
    int4 h[8];                           // eight loads in flight, for any number of CTAs
#pragma unroll
    for (int j = 0; j < 8; ++j)
      h[j] = c0 + 16 * j < (int)gridDim.x ? *reinterpret_cast<const int4*>(hist + (long long)(c0 + 16 * j) * RO_E + e)
                                          : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int m = c0 + 16 * j < (int)blockIdx.x ? -1 : 0;
      all.x += h[j].x; all.y += h[j].y; all.z += h[j].z; all.w += h[j].w;
      mine.x += h[j].x & m; mine.y += h[j].y & m; mine.z += h[j].z & m; mine.w += h[j].w & m;
    }
  }
  *reinterpret_cast<int4*>(&part[0][p][e]) = all;
  *reinterpret_cast<int4*>(&part[1][p][e]) = mine;
  ro_count(s, idx, a0, a1, E, status);
  __syncthreads();
  if (tid < RO_E) {
    int a = 0, b = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a += part[0][i][tid];
      b += part[1][i][tid];
    }
    s.cnt[tid] = a;
    s.before[tid] = b;
  }
  __syncthreads();
  ro_offsets(s.cnt, E, s.offs);
  __syncthreads();
  if (tid < E) {
    int c = s.offs[tid] + s.before[tid];
    for (int w = 0; w < 8; ++w) {
      const int t = s.wh[w][tid];
      s.wh[w][tid] = c;
      c += t;
    }
  }
  if (blockIdx.x == 0 && tid <= E) offs[tid] = s.offs[tid];
  __syncthreads();
  ro_place(s, idx, a0, a1, E, status, perm, row);
  ro_pads(s.cnt, s.offs, E, rows, perm, blockIdx.x * 256LL + tid, gridDim.x * 256LL);
}

// ---------------------------------------------------------------------------
// rows there and back
// ---------------------------------------------------------------------------
// Padding row i of E * 128 candidates (the last 128 rows of each segment), or
// -1: the rows that no token writes.
__device__ __forceinline__ long long pad_row(long long i, int E, const int* offs, const int* perm, long long rows) {
  const int e = (int)(i >> 7);
  if (e >= E) return -1;
  const long long r = (long long)offs[e + 1] - 128 + (i & 127);
  if (r < 0 || r < offs[e] || r >= rows) return -1;
  return perm[r] < 0 ? r : -1;
}

// A lane's part of a chunk of 256 columns: eight neighbours, or in rows of any
// alignment every 32nd element, so that each access of the warp is one segment.
constexpr int MOVE_STEP = 32;
#define MOVE_COL(VEC) ((VEC) ? lane * 8 : lane)

// A warp holds one token's chunk of 256 columns (8 per lane) and writes it to
// the token's rows: x is read once however many experts take it, which leaves
// the write of the copies as the bound.  The CTAs behind the tokens' write the
// padding rows.
template <class T, int VEC>
__global__ void __launch_bounds__(256) dispatch_k(const T* x, long long ldx, long long tokens, int width, int K,
                                                  int E, const int* offs, const int* perm, const int* row,
                                                  long long rows, T* out, long long ldo, long long tok_ctas) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float zero[8] = {};
  if (blockIdx.x >= tok_ctas) {
    const long long r = pad_row((blockIdx.x - tok_ctas) * 8 + warp, E, offs, perm, rows);
    if (r < 0) return;
    for (int c0 = 256 * (int)blockIdx.y; c0 < width; c0 += 256 * (int)gridDim.y)
      ops_st8<VEC, MOVE_STEP>(out + r * ldo, c0 + MOVE_COL(VEC), width, zero);
    return;
  }
  const long long t = (long long)blockIdx.x * 8 + warp;
  if (t >= tokens) return;
  const int mine = lane < K ? row[t * K + lane] : -1;
  for (int c0 = 256 * (int)blockIdx.y; c0 < width; c0 += 256 * (int)gridDim.y) {
    const int c = c0 + MOVE_COL(VEC);
    Raw8<T> v;
    v.template load<VEC, MOVE_STEP>(x + t * ldx, c, width);
    for (int k = 0; k < K; ++k) {
      const long long r = __shfl_sync(0xffffffffu, mine, k);
      if (r >= 0 && r < rows) v.template store<VEC, MOVE_STEP>(out + r * ldo, c, width);
    }
  }
}

// The same with the row's blocks quantised in registers (a block of 128 lies
// in 16 lanes), once per token.
template <class T, int VEC, int CH>
__global__ void __launch_bounds__(256) dispatch8_k(const T* x, long long ldx, long long tokens, int width, int K,
                                                   int E, const int* offs, const int* perm, const int* row,
                                                   long long rows, uint8_t* q, long long ldq, uint8_t* sc,
                                                   long long lds, long long tok_ctas) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= tok_ctas) {
    const long long r = pad_row((blockIdx.x - tok_ctas) * 8 + warp, E, offs, perm, rows);
    if (r < 0) return;
    for (int c = lane * 8 + 256 * (int)blockIdx.y; c < width; c += 256 * (int)gridDim.y) {
      ops_st_codes<VEC>(q + r * ldq, c, width, make_uint2(0, 0), true);
      if ((lane & 15) == 0) sc[r * lds + (c >> 7)] = 127;
    }
    return;
  }
  const long long t = (long long)blockIdx.x * 8 + warp;
  if (t >= tokens) return;
  int mine = lane < K ? row[t * K + lane] : -1;
  if (mine >= rows) mine = -1;
  for (int c0 = 256 * CH * (int)blockIdx.y; c0 < width; c0 += 256 * CH * (int)gridDim.y) {
    Raw8<T> x8[CH];
#pragma unroll
    for (int h = 0; h < CH; ++h)
      if (c0 + 256 * h < width) x8[h].template load<VEC>(x + t * ldx, c0 + 256 * h + lane * 8, width);
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      const int c = c0 + 256 * h + lane * 8;
      if (c0 + 256 * h >= width) break;
      float v[8];
      uint32_t e;
      x8[h].values(v);
      const uint2 codes = ops_quantise(v, ops_max16(x8[h].top()), &e);
      const bool first = (lane & 15) == 0 && c < width;
      for (int k = 0; k < K; ++k) {
        const int r = __shfl_sync(0xffffffffu, mine, k);
        if (r < 0) continue;
        ops_st_codes<VEC>(q + (long long)r * ldq, c, width, codes, true);
        if (first) sc[(long long)r * lds + (c >> 7)] = (uint8_t)e;
      }
    }
  }
}

// A warp sums one token's row over its slots in order, in fp32.  KM bounds K, CH
// chunks of 256 columns are taken at once: every load of all slots and chunks is
// in flight before the first sum (8 of 16 bytes per lane and more), so that the
// trip for the row numbers is paid once for a whole row.
template <class T, int VEC, int KM, int CH>
__global__ void __launch_bounds__(256) combine_k(const T* y, long long ldy, long long rows, const int* row,
                                                 const float* w, long long tokens, int K, int width, T* out,
                                                 long long ldo) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * 8 + warp;
  if (t >= tokens) return;
  int mine = lane < K ? row[t * K + lane] : -1;
  if (mine >= rows) mine = -1;
  const float wm = lane < K ? (w ? w[t * K + lane] : 1.f) : 0.f;
  for (int c0 = 256 * CH * (int)blockIdx.y; c0 < width; c0 += 256 * CH * (int)gridDim.y) {
    Raw8<T> v[KM][CH];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      const long long r = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
      for (int h = 0; h < CH; ++h)
        if (r >= 0 && c0 + 256 * h < width) v[k][h].template load<VEC, MOVE_STEP>(y + r * ldy, c0 + 256 * h + MOVE_COL(VEC), width);
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (c0 + 256 * h >= width) break;
      float s[8] = {};
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wm, k);
        if (__shfl_sync(0xffffffffu, mine, k) >= 0) {
          float x[8];
          v[k][h].values(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = fmaf(wk, x[i], s[i]);
        }
      }
      ops_st8<VEC, MOVE_STEP>(out + t * ldo, c0 + 256 * h + MOVE_COL(VEC), width, s);
    }
  }
}

// A warp takes one token's whole row: dout is read once for its slots, each
// slot's y row is read for the dot product and its dy row written; CH chunks at
// once as above.  For up to two slots of bf16 that is three, the most that 64
// registers hold (four CTAs on an SM; a fourth chunk takes 78 and leaves three).
// 1 / 2 / 3 / 4 chunks, us for 32768 tokens x 2 of 768 columns and as many bytes
// of others: 256 columns 41 / 50 / 50 / 60, 512: 38.6 / 38.7 / 38.7 / 43, 768: 39.0 /
// 39.5 / 38.3 / 39.1, 1024: 39.2 / 38.4 / 38.9 / 38.3, 2048: 39.6 / 39.1 / 39.0 / 38.7,
// 4096: 41.4 / 39.9 / 40.0 / 39.1.  Up to four slots 2 against 1 or 3: 35.5, 36.8, 38.0
// at 1024; fp32 with two slots 2 against 1 or 3: 38.4, 38.6, 39.4.
template <class T, int VEC, int KM, int CH>
__global__ void __launch_bounds__(256) combine_bwd_k(const T* dout, long long lddo, const T* y, long long ldy,
                                                     const int* offs, const int* perm, const int* row, long long rows,
                                                     const float* w, long long tokens, int K, int E, int width,
                                                     T* dy, long long lddy, float* dw, long long tok_ctas) {
  ops_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float zero[8] = {};
  if (blockIdx.x >= tok_ctas) {
    const long long r = pad_row((blockIdx.x - tok_ctas) * 8 + warp, E, offs, perm, rows);
    if (r < 0) return;
    for (int c0 = 0; c0 < width; c0 += 256) ops_st8<VEC, MOVE_STEP>(dy + r * lddy, c0 + MOVE_COL(VEC), width, zero);
    return;
  }
  const long long t = (long long)blockIdx.x * 8 + warp;
  if (t >= tokens) return;
  int mine = lane < K ? row[t * K + lane] : -1;
  if (mine >= rows) mine = -1;
  const float wm = lane < K ? w[t * K + lane] : 0.f;
  float dot[KM] = {};
  for (int c0 = 0; c0 < width; c0 += 256 * CH) {
    Raw8<T> d8[CH], v8[KM][CH];
#pragma unroll
    for (int h = 0; h < CH; ++h)
      if (c0 + 256 * h < width) d8[h].template load<VEC, MOVE_STEP>(dout + t * lddo, c0 + 256 * h + MOVE_COL(VEC), width);
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      const long long r = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
      for (int h = 0; h < CH; ++h)
        if (r >= 0 && c0 + 256 * h < width) v8[k][h].template load<VEC, MOVE_STEP>(y + r * ldy, c0 + 256 * h + MOVE_COL(VEC), width);
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (c0 + 256 * h >= width) break;
      float d[8];
      d8[h].values(d);
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        const long long r = __shfl_sync(0xffffffffu, mine, k);
        const float wk = __shfl_sync(0xffffffffu, wm, k);
        if (r < 0) continue;
        float o[8], v[8];
        v8[k][h].values(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = wk * d[i];
          dot[k] = fmaf(d[i], v[i], dot[k]);
        }
        ops_st8<VEC, MOVE_STEP>(dy + r * lddy, c0 + 256 * h + MOVE_COL(VEC), width, o);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    float s = dot[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == k && k < K) dw[t * K + k] = s;
  }
}

int route_ok(int64_t tokens, int32_t K, int32_t E) {
  if (tokens < 0 || K < 1 || E < 1) return MT_ERR_ARG;
  if (E > MT_MAX_EXPERTS || K > 8 || K > E || tokens > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  if (tokens * K + (int64_t)E * 128 > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  return MT_OK;
}
int64_t route_rows(int64_t tokens, int32_t K, int32_t E) {
  return (tokens * K + (int64_t)E * 127 + 127) / 128 * 128;
}
// assignments per CTA of the grid
int64_t route_chunk(int64_t n) {
  const int64_t per = (n + RO_GRID - 1) / RO_GRID;
  return (per + RO_CHUNK - 1) / RO_CHUNK * RO_CHUNK;
}
// chunks of 256 columns as a second grid dimension (a CTA walks on from there)
unsigned col_chunks(int64_t width) {
  const int64_t n = (width + 255) / 256;
  return (unsigned)(n < 1024 ? n : 1024);
}

template <class T>
int dispatch_t(const void* x, int64_t ldx, int64_t tokens, int64_t width, int K, int E, const int* offs,
               const int* perm, const int* row, int64_t rows, void* out, int64_t ldo, int vec, cudaStream_t st) {
  const long long tc = (tokens + 7) / 8;
  const dim3 grid((unsigned)(tc + E * 16), col_chunks(width));
  auto k = vec == 2 ? dispatch_k<T, 2> : vec ? dispatch_k<T, 1> : dispatch_k<T, 0>;
  return ops_launch(k, grid, 256, 0, st, 1, (const T*)x, ldx, tokens, (int)width, K, E, offs, perm, row, rows, (T*)out, ldo, tc);
}
template <class T, int VEC>
int dispatch8_t(const void* x, int64_t ldx, int64_t tokens, int K, int E, const int* offs, const int* perm,
                const int* row, const mt_mat8* o, cudaStream_t st) {
  const long long tc = (tokens + 7) / 8;
  // few tokens spread their columns over the grid, many take a row per warp
  constexpr int CH = sizeof(T) == 4 ? 2 : 4;
  const bool wide = tokens * ((o->cols + 255) / 256) > 152 * 16;
  const dim3 grid((unsigned)(tc + E * 16), col_chunks(wide ? (o->cols + CH - 1) / CH : o->cols));
  auto k = wide ? dispatch8_k<T, VEC, CH> : dispatch8_k<T, VEC, 1>;
  return ops_launch(k, grid, 256, 0, st, 1, (const T*)x, ldx, tokens, (int)o->cols, K, E, offs, perm, row, o->rows, (uint8_t*)o->codes,
                          o->ld, (uint8_t*)o->scales, o->lds, tc);
}
template <class T, int VEC>
int combine_t(const void* y, int64_t ldy, int64_t rows, const int* row, const float* w, int64_t tokens, int K,
              int64_t width, void* out, int64_t ldo, cudaStream_t st) {
  // few tokens spread their columns over the grid, many take a row per warp
  constexpr bool F = sizeof(T) == 4;
  const int64_t per = K <= 2 ? (F ? 2 : 4) : K <= 4 ? (F ? 1 : 2) : 1;
  const dim3 grid((unsigned)((tokens + 7) / 8), col_chunks((width + per - 1) / per));
  auto k = K <= 2 ? combine_k<T, VEC, 2, F ? 2 : 4> : K <= 4 ? combine_k<T, VEC, 4, F ? 1 : 2> : combine_k<T, VEC, 8, 1>;
  return ops_launch(k, grid, 256, 0, st, 1, (const T*)y, ldy, rows, row, w, tokens, K, (int)width, (T*)out, ldo);
}
template <class T, int VEC>
int combine_bwd_t(const void* dout, int64_t lddo, const void* y, int64_t ldy, const int* offs, const int* perm,
                  const int* row, int64_t rows, const float* w, int64_t tokens, int K, int E, int64_t width, void* dy,
                  int64_t lddy, float* dw, cudaStream_t st) {
  const long long tc = (tokens + 7) / 8;
  constexpr bool F = sizeof(T) == 4;
  auto k = K <= 2   ? combine_bwd_k<T, VEC, 2, F ? 2 : 3>
           : K <= 4 ? combine_bwd_k<T, VEC, 4, F ? 1 : 2>
                    : combine_bwd_k<T, VEC, 8, 1>;
  return ops_launch(k, (unsigned)(tc + E * 16), 256, 0, st, 1, (const T*)dout, lddo, (const T*)y, ldy, offs, perm, row, rows, w, tokens,
                                             K, E, (int)width, (T*)dy, lddy, dw, tc);
}

// checks of the routing triple as the moves read it
int moves_ok(int64_t tokens, int32_t K, int32_t E, int64_t rows, int64_t width, const void* offs, const void* perm,
             const void* row) {
  const int st = route_ok(tokens, K, E);
  if (st) return st;
  if (rows < 0 || width < 1) return MT_ERR_ARG;
  if (rows > OPS_MAX_ROWS || width > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  if (!offs || !perm || (tokens && !row) || !ops_aligned(offs, 4) || !ops_aligned(perm, 4) || !ops_aligned(row, 4))
    return MT_ERR_ARG;
  // perm and offs were made for this many rows
  return rows == route_rows(tokens, K, E) ? MT_OK : MT_ERR_ARG;
}

}  // namespace

extern "C" {

int64_t mt_route_rows(int64_t n_tokens, int32_t top_k, int32_t n_experts) {
  const int st = route_ok(n_tokens, top_k, n_experts);
  return st ? -st : route_rows(n_tokens, top_k, n_experts);
}

int64_t mt_route_ws_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts) {
  const int st = route_ok(n_tokens, top_k, n_experts);
  if (st) return -st;
  const int64_t n = n_tokens * top_k;
  return n <= RO_CLUSTER ? 16 : (n + route_chunk(n) - 1) / route_chunk(n) * RO_E * 4;
}

int32_t mt_route_order(const int32_t* idx, int64_t n_tokens, int32_t top_k, int32_t n_experts, int32_t* offs,
                       int32_t* perm, int32_t* row, void* ws, int64_t ws_bytes, int32_t* status, void* stream) {
  const int st = route_ok(n_tokens, top_k, n_experts);
  if (st) return st;
  if (!offs || !perm || !status || (n_tokens && (!idx || !row))) return MT_ERR_ARG;
  if (!ops_aligned(idx, 4) || !ops_aligned(offs, 4) || !ops_aligned(perm, 4) || !ops_aligned(row, 4) ||
      !ops_aligned(status, 4))
    return MT_ERR_ARG;
  if (!ws || !ops_aligned(ws, 16)) return MT_ERR_ARG;
  if (ws_bytes < mt_route_ws_bytes(n_tokens, top_k, n_experts)) return MT_ERR_ARENA_SMALL;
  const int64_t n = n_tokens * top_k, rows = route_rows(n_tokens, top_k, n_experts);
  cudaStream_t s = (cudaStream_t)stream;
  if (n <= RO_SMALL) {
    return ops_launch(ro_sort<1>, 1, 1024, 0, s, 1, idx, n, n_experts, rows, offs, perm, row, status);
  }
  if (n <= RO_CLUSTER) {
    // sixteen CTAs per cluster are an opt-in of this architecture
    if (cudaFuncSetAttribute(ro_sort<RO_CTAS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return MT_ERR_LAUNCH;
    }
    return ops_launch(ro_sort<RO_CTAS>, RO_CTAS, 1024, 0, s, RO_CTAS, idx, n, n_experts, rows, offs, perm, row, status);
  }
  const int64_t chunk = route_chunk(n);
  const unsigned chunks = (unsigned)((n + chunk - 1) / chunk);
  const int rc = ops_launch(ro_hist, chunks, 256, 0, s, 1, idx, n, chunk, n_experts, (int*)ws, status);
  if (rc) return rc;
  return ops_launch(ro_scatter, chunks, 256, 0, s, 1, idx, n, chunk, n_experts, rows, (const int*)ws, offs, perm,
                    row, status);
}

int32_t mt_dispatch(const void* x, int32_t dtype, int64_t ldx, int64_t n_tokens, int64_t width, int32_t top_k,
                    int32_t n_experts, const int32_t* offs, const int32_t* perm, const int32_t* row, int64_t rows,
                    void* out, int64_t ldo, void* stream) {
  const int st = moves_ok(n_tokens, top_k, n_experts, rows, width, offs, perm, row);
  if (st) return st;
  if (!ops_dtype_ok(dtype) || !ops_mat_ok(out, dtype, ldo, width)) return MT_ERR_ARG;
  if (n_tokens == 0) return MT_OK;
  if (!ops_mat_ok(x, dtype, ldx, width)) return MT_ERR_ARG;
  const int vec = ops_mode(ops_least(ops_vec(x, dtype, ldx), ops_vec(out, dtype, ldo)), width, 256);
  auto f = dtype == MT_DT_FP32 ? dispatch_t<float> : dispatch_t<__nv_bfloat16>;
  return f(x, ldx, n_tokens, width, top_k, n_experts, offs, perm, row, rows, out, ldo, vec, (cudaStream_t)stream);
}

int32_t mt_dispatch8(const void* x, int32_t dtype, int64_t ldx, int64_t n_tokens, int32_t top_k, int32_t n_experts,
                     const int32_t* offs, const int32_t* perm, const int32_t* row, const mt_mat8* out, void* stream) {
  if (!ops_mat8_ok(out) || out->block_rows != 1 || out->batch != 1 || out->halves) return MT_ERR_ARG;
  const int st = moves_ok(n_tokens, top_k, n_experts, out->rows, out->cols, offs, perm, row);
  if (st) return st;
  if (!ops_dtype_ok(dtype)) return MT_ERR_ARG;
  if (n_tokens == 0) return MT_OK;
  if (!ops_mat_ok(x, dtype, ldx, out->cols)) return MT_ERR_ARG;
  const int vec = ops_mode(ops_vec(x, dtype, ldx), out->cols, 256);
  auto f = dtype == MT_DT_FP32
               ? (vec == 2 ? dispatch8_t<float, 2> : vec ? dispatch8_t<float, 1> : dispatch8_t<float, 0>)
               : (vec == 2 ? dispatch8_t<__nv_bfloat16, 2> : vec ? dispatch8_t<__nv_bfloat16, 1> : dispatch8_t<__nv_bfloat16, 0>);
  return f(x, ldx, n_tokens, top_k, n_experts, offs, perm, row, out, (cudaStream_t)stream);
}

int32_t mt_combine(const void* y, int32_t dtype, int64_t ldy, int64_t rows, const int32_t* row, const float* w,
                   int64_t n_tokens, int32_t top_k, int64_t width, void* out, int64_t ldo, void* stream) {
  const int st = route_ok(n_tokens, top_k, MT_MAX_EXPERTS);
  if (st) return st;
  if (rows < 0 || width < 1 || !ops_dtype_ok(dtype)) return MT_ERR_ARG;
  if (rows > OPS_MAX_ROWS || width > OPS_MAX_ROWS) return MT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MT_OK;
  if (!row || !ops_aligned(row, 4) || !ops_aligned(w, 4)) return MT_ERR_ARG;
  if (!ops_mat_ok(y, dtype, ldy, width) || !ops_mat_ok(out, dtype, ldo, width)) return MT_ERR_ARG;
  const int vec = ops_mode(ops_least(ops_vec(y, dtype, ldy), ops_vec(out, dtype, ldo)), width, 256);
  auto f = dtype == MT_DT_FP32
               ? (vec == 2 ? combine_t<float, 2> : vec ? combine_t<float, 1> : combine_t<float, 0>)
               : (vec == 2 ? combine_t<__nv_bfloat16, 2> : vec ? combine_t<__nv_bfloat16, 1> : combine_t<__nv_bfloat16, 0>);
  return f(y, ldy, rows, row, w, n_tokens, top_k, width, out, ldo, (cudaStream_t)stream);
}

int32_t mt_combine_bwd(const void* dout, int32_t dtype, int64_t lddo, const void* y, int64_t ldy, const int32_t* offs,
                       const int32_t* perm, const int32_t* row, int64_t rows, const float* w, int64_t n_tokens,
                       int32_t top_k, int32_t n_experts, int64_t width, void* dy, int64_t lddy, float* dw,
                       void* stream) {
  const int st = moves_ok(n_tokens, top_k, n_experts, rows, width, offs, perm, row);
  if (st) return st;
  if (!ops_dtype_ok(dtype)) return MT_ERR_ARG;
  if (n_tokens == 0) return MT_OK;
  if (!w || !dw || !ops_aligned(w, 4) || !ops_aligned(dw, 4)) return MT_ERR_ARG;
  if (!ops_mat_ok(dout, dtype, lddo, width) || !ops_mat_ok(y, dtype, ldy, width) || !ops_mat_ok(dy, dtype, lddy, width))
    return MT_ERR_ARG;
  const int vec = ops_mode(ops_least(ops_vec(dout, dtype, lddo), ops_least(ops_vec(y, dtype, ldy), ops_vec(dy, dtype, lddy))), width, 256);
  auto f = dtype == MT_DT_FP32
               ? (vec == 2 ? combine_bwd_t<float, 2> : vec ? combine_bwd_t<float, 1> : combine_bwd_t<float, 0>)
               : (vec == 2 ? combine_bwd_t<__nv_bfloat16, 2>
                  : vec    ? combine_bwd_t<__nv_bfloat16, 1>
                           : combine_bwd_t<__nv_bfloat16, 0>);
  return f(dout, lddo, y, ldy, offs, perm, row, rows, w, n_tokens, top_k, n_experts, width, dy, lddy, dw,
           (cudaStream_t)stream);
}

}  // extern "C"
