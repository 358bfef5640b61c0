// gemm8.cu - products of 8-bit matrices with a scale per block of 128
// (mt_gemm8, mt_gemm8_reduce) on tcgen05 tensor cores.
//
//   C[m,n] = sum over blocks b of 2^(ea[m,b] + eb[n,b]) * (qa[m,b,:] . qb[n,b,:])
//
// One persistent CTA per SM walks 128 x BN tiles of C.  Per tile and block of
// 128 along the reduction:
//   warp 0      TMA producer: one 128-byte-swizzled box of A and one of B per
//               block into a ring of stages;
//   warp 1      four tcgen05.mma kind::f8f6f4 (128 x BN x 32) into one of two
//               TMEM accumulators, started from zero for each block;
//   warps 2..9  read the block's sums from TMEM and add them, scaled, to fp32
//               registers (two-wide FMAs), while the tensor cores run the next
//               block; after the last block they store the tile.
// The scale is applied outside the tensor core because it is free there: 128
// blocks of K hold the MMA for 4 * BN * 128 / 1024 cycles, in which the eight
// warps read and scale 16 K values.  It also keeps the sum over blocks in
// rounded fp32 additions.
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "gemm_tc.cuh"
#include "ops8.cuh"
#include "tmaps.h"

namespace {

constexpr int G8_THREADS = 320;
constexpr int G8_STAGES = 4;
constexpr int G8_A_BYTES = 128 * 128;
constexpr int G8_WIN = 4096;                 // epilogue window per warp: 32 rows x 128 bytes
constexpr long long G8_TIMEOUT_NS = 2000000000LL;
enum { G8_DENSE = 0, G8_ROWS = 1, G8_REDUCE = 2 };

// shared memory below the stages (offsets from the base)
constexpr int G8_TMEM = 0;
constexpr int G8_ABORT = 4;
constexpr int G8_BAR = 16;                   // full[4], empty[4], tfull[2], tempty[2]
constexpr int G8_OFFS = 160;                 // segment starts: 65 ints
constexpr int G8_SB = 512;                   // column scales of two blocks: 2 x 256 floats
constexpr int G8_DATA = 3072;

constexpr int g8_smem(int bn) { return G8_DATA + G8_STAGES * (G8_A_BYTES + bn * 128) + 8 * G8_WIN; }
static_assert(g8_smem(256) <= 232448, "shared memory exceeds 227 KB");

struct G8Args {
  CUtensorMap a, b, c;
  const uint8_t* sa;
  const uint8_t* sb;
  const int* offs;
  void* out;
  int* status;
  long long ldsa, ldsb, ldc;
  int M, N, K, nseg, mode, mt, nt, ntiles, accumulate, tma_out;
};

// 2^(byte a + byte b - 254), 0 below 2^-126 and 2^127 above
__device__ __forceinline__ float g8_scale(int a, int b) {
  int e = a + b - 127;
  e = e < 1 ? 0 : e > 254 ? 254 : e;
  return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ void g8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void g8_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   (unsigned long long)map),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void g8_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   (unsigned long long)map),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Bounded wait that also ends when another role of the CTA gave up.
__device__ __forceinline__ bool g8_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if ((long long)(globaltimer() - t0) > G8_TIMEOUT_NS) {
      *abort = 1;
      if (atomicCAS(status, 0, (int)MT_ERR_DEVICE_TIMEOUT) == 0) status[1] = site;
      return false;
    }
  }
  return true;
}

struct G8Tile {
  int m0, n0, seg, k0, nkb;      // first row and column of C, segment, first element and blocks of K
};
// Tile t, or false where the segments leave none.  Columns go fastest: the
// CTAs running at one time share rows of A and the (small) B in L2.
template <int BN>
__device__ __forceinline__ bool g8_tile(const G8Args& g, const int* offs, int t, G8Tile& ti) {
  const int per = g.mt * g.nt;
  ti.seg = 0;
  if (g.mode == G8_REDUCE) {
    ti.seg = t / per;
    t -= ti.seg * per;
  }
  ti.m0 = (t / g.nt) * 128;
  ti.n0 = (t % g.nt) * BN;
  ti.k0 = 0;
  ti.nkb = (g.K + 127) >> 7;
  if (g.mode == G8_ROWS) {
    if (ti.m0 >= offs[g.nseg]) return false;
    int lo = 0, hi = g.nseg - 1;           // last segment that starts at or before m0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offs[mid] <= ti.m0) lo = mid;
      else hi = mid - 1;
    }
    ti.seg = lo;
  } else if (g.mode == G8_REDUCE) {
    ti.k0 = offs[ti.seg];
    ti.nkb = (offs[ti.seg + 1] - ti.k0 + 127) >> 7;
  }
  return true;
}

template <class CT>
__device__ __forceinline__ void g8_put(uint32_t win, int lane, const float* v);
template <>
__device__ __forceinline__ void g8_put<float>(uint32_t win, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts128(win + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
           __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
}
template <>
__device__ __forceinline__ void g8_put<__nv_bfloat16>(uint32_t win, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts128(win + lane * 128 + ((j ^ (lane & 7)) << 4), ops_bf2(v[8 * j], v[8 * j + 1]),
           ops_bf2(v[8 * j + 2], v[8 * j + 3]), ops_bf2(v[8 * j + 4], v[8 * j + 5]),
           ops_bf2(v[8 * j + 6], v[8 * j + 7]));
}

// BN: columns of a tile.  BCOL: B has a scale per row (column of C) instead of
// one per 128.  CT: type of C.
template <int BN, bool BCOL, class CT>
__global__ void __launch_bounds__(G8_THREADS, 1) gemm8_k(const __grid_constant__ G8Args g) {
  extern __shared__ __align__(1024) char gen[];
  constexpr int STAGE = G8_A_BYTES + BN * 128;
  constexpr int HALF = BN == 64 ? 64 : BN / 2;        // columns per epilogue warp (a window holds 64 of bf16)
  constexpr int EW = 4 * (BN / HALF);                 // epilogue warps
  constexpr int CW = 128 / (int)sizeof(CT);           // columns of a window
  const uint32_t base = smem_u32(gen);
  if (base & 1023) {                                  // swizzled tiles start on 1024-byte boundaries
    if (threadIdx.x == 0 && atomicCAS(g.status, 0, (int)MT_ERR_LAUNCH) == 0) g.status[1] = SITE_TC_ALIGN;
    return;
  }
  volatile int* abort = reinterpret_cast<volatile int*>(gen + G8_ABORT);
  int* offs = reinterpret_cast<int*>(gen + G8_OFFS);
  float* sbuf = reinterpret_cast<float*>(gen + G8_SB);
  const uint32_t full = base + G8_BAR, empty = full + 8 * G8_STAGES, tfull = empty + 8 * G8_STAGES, tempty = tfull + 16;
  const uint32_t stages = base + G8_DATA;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < G8_STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, EW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // segment starts, kept inside the operands and on block boundaries whatever
  // they hold (a TMA coordinate has to be a multiple of 16)
  if (g.mode != G8_DENSE && tid <= g.nseg) {
    const int lim = g.mode == G8_ROWS ? (g.M + 127) & ~127 : g.K;
    int v = __ldg(g.offs + tid) & ~127;
    v = v < 0 ? 0 : v > lim ? lim : v;
    offs[tid] = v & ~127;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + G8_TMEM), "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gen + G8_TMEM);

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < g.ntiles && ok; t += gridDim.x) {
        G8Tile ti;
        if (!g8_tile<BN>(g, offs, t, ti)) continue;
        const int by = (g.mode == G8_ROWS ? ti.seg * g.N : 0) + ti.n0;
        for (int kb = 0; kb < ti.nkb; ++kb, ++it) {
          const int s = it % G8_STAGES;
          if (it >= G8_STAGES && !g8_wait(empty + 8 * s, (it / G8_STAGES - 1) & 1, abort, g.status, SITE_TC_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sm = stages + s * STAGE;
          mbar_expect_tx(full + 8 * s, STAGE);
          tma_load_2d(sm, &g.a, ti.k0 + kb * 128, ti.m0, full + 8 * s);
          tma_load_2d(sm + G8_A_BYTES, &g.b, ti.k0 + kb * 128, by, full + 8 * s);
        }
      }
      if (!ok)       // let the copies in flight land before the CTA leaves
        for (int i = it > G8_STAGES ? it - G8_STAGES : 0; i < it; ++i) {
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(full + 8 * (i % G8_STAGES), (i / G8_STAGES) & 1) &&
                 (long long)(globaltimer() - t0) < G8_TIMEOUT_NS) {
          }
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // e4m3 x e4m3 -> fp32, both K-major
      const uint32_t idesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < g.ntiles && ok; t += gridDim.x) {
        G8Tile ti;
        if (!g8_tile<BN>(g, offs, t, ti)) continue;
        for (int kb = 0; kb < ti.nkb; ++kb, ++it) {
          const int s = it % G8_STAGES, d = it & 1;
          if (!g8_wait(full + 8 * s, (it / G8_STAGES) & 1, abort, g.status, SITE_TC_FULL) ||
              (it >= 2 && !g8_wait(tempty + 8 * d, (it / 2 - 1) & 1, abort, g.status, SITE_TC_ACC_EMPTY))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sm = stages + s * STAGE;
          const uint64_t ad = sdesc(sm, 16, 1024), bd = sdesc(sm + G8_A_BYTES, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            g8_mma(tmem + d * BN, sdesc_add(ad, 32 * k), sdesc_add(bd, 32 * k), idesc, k > 0);
          mma_commit(empty + 8 * s);
          mma_commit(tfull + 8 * d);
        }
      }
      // every issued product has arrived before the TMEM is freed
      const unsigned long long t0 = globaltimer();
      while (it > 0 && !mbar_try_wait(tfull + 8 * ((it - 1) & 1), ((it - 1) / 2) & 1) &&
             (long long)(globaltimer() - t0) < G8_TIMEOUT_NS) {
      }
    }
  } else if (warp < 2 + EW) {
    const int et = tid - 64, ew = warp - 2, quad = warp & 3, half = ew >> 2;
    const uint32_t win = stages + G8_STAGES * STAGE + ew * G8_WIN;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + half * HALF;
    const int nrb = (g.N + 127) >> 7;
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < g.ntiles; t += gridDim.x) {
      G8Tile ti;
      if (!g8_tile<BN>(g, offs, t, ti)) continue;
      const int row = ti.m0 + quad * 32 + lane, col = ti.n0 + half * HALF;
      const uint8_t* pa = g.sa + (long long)(row < g.M ? row : g.M - 1) * g.ldsa + (ti.k0 >> 7);
      const uint8_t* pb;
      if (BCOL) {
        const int c = ti.n0 + (et < BN ? et : 0);
        pb = g.sb + ((long long)(g.mode == G8_ROWS ? ti.seg : 0) * g.N + (c < g.N ? c : g.N - 1)) * g.ldsb + (ti.k0 >> 7);
      } else {
        const int rb = col >> 7;
        pb = g.sb + ((long long)(g.mode == G8_ROWS ? ti.seg : 0) * nrb + (rb < nrb ? rb : nrb - 1)) * g.ldsb + (ti.k0 >> 7);
      }
      uint64_t acc[HALF / 2];
#pragma unroll
      for (int i = 0; i < HALF / 2; ++i) acc[i] = 0;
      int a1 = ti.nkb ? __ldg(pa) : 0, b1 = ti.nkb ? __ldg(pb) : 0;
      for (int kb = 0; kb < ti.nkb; ++kb, ++it) {
        const int a0 = a1, b0 = b1, d = it & 1;
        if (kb + 1 < ti.nkb) {
          a1 = __ldg(pa + kb + 1);
          b1 = __ldg(pb + kb + 1);
        }
        if (BCOL) {
          // per-column scales of this block; the other half of the buffer may
          // still be read for the block before
          if (et < BN) sbuf[d * 256 + et] = g8_scale(b0, 127);
          asm volatile("bar.sync 1, %0;" ::"n"(32 * EW) : "memory");
        }
        const float s = BCOL ? g8_scale(a0, 127) : g8_scale(a0, b0);
        const uint64_t s2 = f2(s, s);
        if (!g8_wait(tfull + 8 * d, (it / 2) & 1, abort, g.status, SITE_TC_ACC_FULL)) ok = false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HALF; c += 32) {
          float v[32];
          tmem_ld32(trow + d * BN + c, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            if (BCOL) {
              const float4 f = *reinterpret_cast<const float4*>(sbuf + d * 256 + half * HALF + c + i);
              acc[(c + i) / 2] = fma2(mul2(f2(v[i], v[i + 1]), f2(f.x, f.y)), s2, acc[(c + i) / 2]);
              acc[(c + i) / 2 + 1] = fma2(mul2(f2(v[i + 2], v[i + 3]), f2(f.z, f.w)), s2, acc[(c + i) / 2 + 1]);
            } else {
              acc[(c + i) / 2] = fma2(f2(v[i], v[i + 1]), s2, acc[(c + i) / 2]);
              acc[(c + i) / 2 + 1] = fma2(f2(v[i + 2], v[i + 3]), s2, acc[(c + i) / 2 + 1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty + 8 * d);
      }
      // after a wait that gave up every later one ends at once: walk on to keep
      // the named barriers paired, and store nothing more
      ok = !__any_sync(0xffffffffu, !ok);
      if (!ok || (ti.nkb == 0 && g.accumulate)) continue;
      const int z = g.mode == G8_REDUCE ? ti.seg : 0, row0 = ti.m0 + quad * 32;
#pragma unroll
      for (int c = 0; c < HALF; c += CW) {
        float v[CW];
#pragma unroll
        for (int i = 0; i < CW; i += 2) unf2(acc[(c + i) / 2], v[i], v[i + 1]);
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        g8_put<CT>(win, lane, v);
        if (col + c >= g.N || row0 >= g.M) continue;
        if (g.tma_out) {
          fence_smem_async();
          __syncwarp();
          if (lane == 0) {
            if (sizeof(CT) == 4 && g.accumulate) g8_add_3d(&g.c, win, col + c, row0, z);
            else g8_store_3d(&g.c, win, col + c, row0, z);
            bulk_commit();
          }
        } else {
          // rows of any alignment: the window is read back a row at a time
          __syncwarp();
          const int rows = g.M - row0 < 32 ? g.M - row0 : 32;
          const char* w = gen + (win - base);
          for (int r = 0; r < rows; ++r) {
            CT* dst = reinterpret_cast<CT*>(g.out) + ((long long)z * g.M + row0 + r) * g.ldc + col + c;
#pragma unroll
            for (int i = 0; i < CW; i += 32) {
              const int x = i + lane, off = x * (int)sizeof(CT);
              if (col + c + x < g.N) {
                const CT e = *reinterpret_cast<const CT*>(w + r * 128 + ((((off >> 4) ^ (r & 7))) << 4) + (off & 15));
                if constexpr (sizeof(CT) == 4) dst[x] = g.accumulate ? dst[x] + e : e;
                else dst[x] = e;
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct DevInfo {
  int sms = 0;
  bool prepared[12] = {};
};
std::mutex g_mu;
DevInfo g_dev[64];

typedef void (*G8Kernel)(G8Args);
template <int BN>
G8Kernel kernel_of(bool bcol, bool f32) {
  return bcol ? (f32 ? (G8Kernel)gemm8_k<BN, true, float> : (G8Kernel)gemm8_k<BN, true, __nv_bfloat16>)
              : (f32 ? (G8Kernel)gemm8_k<BN, false, float> : (G8Kernel)gemm8_k<BN, false, __nv_bfloat16>);
}

int device_info(int* sms, int* dev) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= 64) return MT_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[*dev];
  if (!d.sms && cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_CUDA;
  }
  *sms = d.sms;
  return MT_OK;
}

int launch(G8Args& g, const mt_mat8* a, const mt_mat8* b, int64_t segs, bool f32, cudaStream_t st) {
  int sms = 0, dev = 0;
  int rc = device_info(&sms, &dev);
  if (rc) return rc;
  const int batch = g.mode == G8_REDUCE ? g.nseg : 1;
  g.mt = (g.M + 127) / 128;
  // Widest tile that still gives every SM one (wider tiles load less per FLOP,
  // narrower ones spread a small product over more SMs).
  int bn = 256;
  while (bn > 64 && ((int64_t)g.mt * ((g.N + bn - 1) / bn) * batch < sms || g.N <= bn / 2)) bn /= 2;
  g.nt = (g.N + bn - 1) / bn;
  const int64_t tiles = (int64_t)g.mt * g.nt * batch;
  if (tiles > 0x7fffffff) return MT_ERR_UNSUPPORTED;
  g.ntiles = (int)tiles;
  const bool bcol = b->block_rows == 1;
  rc = mt_encode_map(&g.a, MT_MAP_U8, a->codes, a->cols, a->rows, 1, a->ld, 0, 128, 128);
  if (rc == MT_OK) rc = mt_encode_map(&g.b, MT_MAP_U8, b->codes, b->cols, b->rows * segs, 1, b->ld, 0, 128, bn);
  const int es = f32 ? 4 : 2;
  g.tma_out = ops_aligned(g.out, 16) && g.ldc * es % 16 == 0;
  if (rc == MT_OK && g.tma_out)
    rc = mt_encode_map(&g.c, f32 ? MT_MAP_F32 : MT_MAP_BF16, g.out, g.N, g.M, batch, g.ldc * es, g.ldc * es * g.M,
                       128 / es, 32);
  if (rc != MT_OK) return rc;
  const int which = (bn == 256 ? 0 : bn == 128 ? 4 : 8) + (bcol ? 2 : 0) + (f32 ? 1 : 0);
  G8Kernel k = bn == 256 ? kernel_of<256>(bcol, f32) : bn == 128 ? kernel_of<128>(bcol, f32) : kernel_of<64>(bcol, f32);
  const int smem = g8_smem(bn);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_dev[dev].prepared[which]) {
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return MT_ERR_LAUNCH;
      }
      g_dev[dev].prepared[which] = true;
    }
  }
  k<<<(unsigned)(tiles < sms ? tiles : sms), G8_THREADS, smem, st>>>(g);
  return ops_launched();
}

bool operand_ok(const mt_mat8* m) { return ops_mat8_ok(m) && !m->halves; }

}  // namespace

extern "C" {

int32_t mt_gemm8(const mt_mat8* a, const mt_mat8* b, const int32_t* offs, int32_t n_seg, void* c, int32_t dtype,
                 int64_t ldc, int32_t accumulate, int32_t* status, void* stream) {
  if (!operand_ok(a) || !operand_ok(b) || a->block_rows != 1 || a->batch != 1 || a->cols != b->cols) return MT_ERR_ARG;
  if (!ops_dtype_ok(dtype) || (accumulate != 0 && accumulate != 1) || (accumulate && dtype != MT_DT_FP32))
    return MT_ERR_ARG;
  if (offs ? (n_seg < 1 || b->batch != n_seg) : (n_seg != 0 || b->batch != 1)) return MT_ERR_ARG;
  if (n_seg > MT_MAX_EXPERTS) return MT_ERR_UNSUPPORTED;
  if (!status || !ops_aligned(status, 4) || !ops_aligned(offs, 4)) return MT_ERR_ARG;
  if (a->rows == 0 || b->rows == 0) return MT_OK;
  if (!ops_mat_ok(c, dtype, ldc, b->rows)) return MT_ERR_ARG;
  G8Args g;
  memset(&g, 0, sizeof(g));
  g.sa = (const uint8_t*)a->scales; g.sb = (const uint8_t*)b->scales;
  g.offs = offs; g.out = c; g.status = status;
  g.ldsa = a->lds; g.ldsb = b->lds; g.ldc = ldc;
  g.M = (int)a->rows; g.N = (int)b->rows; g.K = (int)a->cols;
  g.nseg = n_seg; g.mode = offs ? G8_ROWS : G8_DENSE; g.accumulate = accumulate;
  return launch(g, a, b, b->batch, dtype == MT_DT_FP32, (cudaStream_t)stream);
}

int32_t mt_gemm8_reduce(const mt_mat8* a, const mt_mat8* b, const int32_t* offs, int32_t n_seg, float* c, int64_t ldc,
                        int32_t accumulate, int32_t* status, void* stream) {
  if (!operand_ok(a) || !operand_ok(b) || a->block_rows != 1 || b->block_rows != 1 || a->batch != 1 || b->batch != 1 ||
      a->cols != b->cols)
    return MT_ERR_ARG;
  if (!offs || n_seg < 1 || (accumulate != 0 && accumulate != 1)) return MT_ERR_ARG;
  if (n_seg > MT_MAX_EXPERTS) return MT_ERR_UNSUPPORTED;
  if (!status || !ops_aligned(status, 4) || !ops_aligned(offs, 4)) return MT_ERR_ARG;
  if (a->rows == 0 || b->rows == 0) return MT_OK;
  if (!ops_mat_ok(c, MT_DT_FP32, ldc, b->rows)) return MT_ERR_ARG;
  G8Args g;
  memset(&g, 0, sizeof(g));
  g.sa = (const uint8_t*)a->scales; g.sb = (const uint8_t*)b->scales;
  g.offs = offs; g.out = c; g.status = status;
  g.ldsa = a->lds; g.ldsb = b->lds; g.ldc = ldc;
  g.M = (int)a->rows; g.N = (int)b->rows; g.K = (int)a->cols;
  g.nseg = n_seg; g.mode = G8_REDUCE; g.accumulate = accumulate;
  return launch(g, a, b, 1, true, (cudaStream_t)stream);
}

}  // extern "C"
