// gemm8.cu - products of 8-bit matrices with a scale per block of 128
// (mt_gemm8, mt_gemm8_reduce) on tcgen05 tensor cores.
//
//   C[m,n] = sum over blocks b of 2^(ea[m,b] + eb[n,b]) * (qa[m,b,:] . qb[n,b,:])
//
// The scales are powers of two with the byte encoding that the block-scaled
// products of this architecture read (one byte per row and 32 of K): the byte
// of a block of 128 serves its four MMAs, the tensor core applies it exactly,
// and the sums stay in TMEM over the whole reduction.
//
// One persistent CTA per SM walks 128 x BN tiles of C:
//   warp 0      TMA producer: one 128-byte-swizzled box of A and one of B per
//               block of 128 into a ring of stages;
//   warp 1      per block four tcgen05.mma kind::mxf8f6f4 (128 x BN x 32);
//   warps 2, 3  gather the scale bytes of A and B, four blocks at a time, and copy
//               them from shared memory to one of four places in TMEM, ahead of
//               the products;
//   warps 4..11 read a finished tile into registers (which frees the accumulator
//               for the next tile), round it and store it by bulk copies.
// TMEM additions cut their result off instead of rounding it (measured: 3e-7 of
// the result after 4096 of K, 8e-6 after 32768, where fp32 additions stay at
// 1e-7), so every 4096 of K the sums are read and added up in registers.
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "gemm_tc.cuh"
#include "ops8.cuh"
#include "tmaps.h"

namespace {

constexpr int G8_THREADS = 384;
constexpr int G8_REGS = 168, G8_REGS_LOAD = 88, G8_REGS_EPI = 208;   // at launch; after the split
static_assert(G8_REGS_LOAD + 2 * G8_REGS_EPI <= 3 * G8_REGS, "register split exceeds the launch's registers");
constexpr int G8_A_BYTES = 128 * 128;
constexpr int G8_WIN = 4096;                 // epilogue window per warp: 32 rows x 128 bytes
constexpr int G8_STAGES = 4;
constexpr long long G8_TIMEOUT_NS = 4000000000LL;   // the update's default bound
enum { G8_DENSE = 0, G8_ROWS = 1, G8_REDUCE = 2 };

constexpr int G8_CHUNK = 32;                 // blocks summed in TMEM
constexpr int G8_SLOTS = 4;                  // groups of four blocks whose scales TMEM holds

// shared memory below the stages (offsets from the base): TMEM address, abort
// flag, mbarriers, segment starts, scale bytes of one group
constexpr int G8_TMEM = 0;
constexpr int G8_ABORT = 4;
constexpr int G8_BAR = 8;                    // full[4] empty[4] tfull[2] tempty[2] sready[4] sfree[4] sa end
constexpr int G8_NBAR = 2 * G8_STAGES + 4 + 2 * G8_SLOTS + 2;
constexpr int G8_OFFS = G8_BAR + 8 * G8_NBAR;
constexpr int G8_SFA = (G8_OFFS + 4 * (MT_MAX_EXPERTS + 1) + 15) & ~15;   // 128 rows: word of row m at (m % 32) * 16 + (m / 32) * 4
constexpr int G8_SFB = G8_SFA + 512;         // two times 128 rows
constexpr int G8_DATA = 2048;
static_assert(G8_SFB + 1024 <= G8_DATA, "scale bytes exceed their space");

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
  int M, N, K, nseg, mode, mt, nt, ntiles, accumulate, tma_out, words_a, words_b;
};

// One block of 128: D (+)= (A * 2^sa) (B * 2^sb)^T in four MMAs of 128 x N x 32,
// scale bytes in TMEM, and the arrival on `bar` when they are done.  The whole
// converged warp walks the issue loop, so that descriptors are warp-uniform
// values, and one elected lane issues.  The loop around it is as short as it can
// be: a warp alone issues an instruction every five cycles or so, and a block's
// products take 513 cycles (at BN 256).
__device__ __forceinline__ void g8_mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                             uint32_t sb, uint32_t acc, uint32_t bar) {
#define G8_MMA "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 l;\n\t.reg .b64 a, b;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t" G8_MMA
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t" G8_MMA
      "[%0], a, b, %3, [%4], [%5], q;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t" G8_MMA
      "[%0], a, b, %3, [%4], [%5], q;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t" G8_MMA
      "[%0], a, b, %3, [%4], [%5], q;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(bar)
      : "memory");
#undef G8_MMA
}
// 32 rows x 16 bytes of shared memory to four TMEM columns, repeated in the four lane groups
__device__ __forceinline__ void g8_copy_scales(uint32_t taddr, uint32_t saddr) {
  // no swizzle: 8 rows x 16 bytes contiguous, the next 8 rows 128 bytes on
  const uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 l;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(d)
      : "memory");
}
// C is written once and not read here: evicted first, it leaves A and B in L2
// (54 -> 51.5 us at the output head)
__device__ __forceinline__ void g8_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(
          (unsigned long long)map),
      "r"(src), "r"(x), "r"(y), "r"(z), "l"(l2_evict_first())
      : "memory");
}
__device__ __forceinline__ void g8_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   (unsigned long long)map),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Bounded wait that also ends when another role of the CTA gave up.  The clock
// and the flag are looked at every 64 polls: reading the global timer between
// two polls delayed each hand-off by several hundred cycles.
__device__ __forceinline__ bool g8_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status, int site) {
  unsigned long long t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if (n & 63) continue;
    if (*abort) return false;
    const unsigned long long t = globaltimer();
    if (!t0) t0 = t;
    if ((long long)(t - t0) > G8_TIMEOUT_NS) {
      *abort = 1;
      if (atomicCAS(status, 0, (int)MT_ERR_DEVICE_TIMEOUT) == 0) status[1] = site;
      return false;
    }
  }
  return true;
}

// The same for a converged warp, which goes on only together.
__device__ __forceinline__ bool g8_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, int* status, int site) {
  return __all_sync(0xffffffffu, g8_wait(bar, parity, abort, status, site));
}

// 32 consecutive fp32 columns of this thread's TMEM lane: issue, and wait for
// every read issued so far (the registers pass through the wait, so that no
// use of them moves before it).
__device__ __forceinline__ void g8_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void g8_ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

struct G8Tile {
  int m0, n0, seg, k0, nkb;      // first row and column of C, segment, first element and blocks of K
};
// Tiles in use: all of them, or those from the first segment's start to the last
// one's end.
__device__ __forceinline__ int g8_first(const G8Args& g, const int* offs) {
  return g.mode == G8_ROWS ? (offs[0] >> 7) * g.nt : 0;
}
__device__ __forceinline__ int g8_tiles(const G8Args& g, const int* offs) {
  if (g.mode != G8_ROWS) return g.ntiles;
  const int n = ((offs[g.nseg] + 127) >> 7) * g.nt;
  return n < g.ntiles ? n : g.ntiles;
}
// Blocks of K in tile t (0: an empty segment).
__device__ __forceinline__ int g8_blocks(const G8Args& g, const int* offs, int t) {
  if (g.mode != G8_REDUCE) return (g.K + 127) >> 7;
  const int seg = t / (g.mt * g.nt), n = offs[seg + 1] - offs[seg];
  return n > 0 ? (n + 127) >> 7 : 0;
}
// Columns go fastest: the CTAs running at one time share rows of A and the
// (small) B in L2.
template <int BN>
__device__ __forceinline__ G8Tile g8_tile(const G8Args& g, const int* offs, int t) {
  G8Tile ti;
  ti.nkb = g8_blocks(g, offs, t);
  ti.seg = 0;
  ti.k0 = 0;
  if (g.mode == G8_REDUCE) {
    ti.seg = t / (g.mt * g.nt);
    t -= ti.seg * g.mt * g.nt;
    ti.k0 = offs[ti.seg];
  }
  ti.m0 = (t / g.nt) * 128;
  ti.n0 = (t % g.nt) * BN;
  if (g.mode == G8_ROWS) {
    int lo = 0, hi = g.nseg - 1;           // last segment that starts at or before m0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offs[mid] <= ti.m0) lo = mid;
      else hi = mid - 1;
    }
    ti.seg = lo;
  }
  return ti;
}

// One window of this thread's row (128 bytes) into shared memory, chunks
// swizzled as the bulk store's map expects.
template <class CT>
__device__ __forceinline__ void g8_put(uint32_t win, int lane, const uint32_t* v);
template <>
__device__ __forceinline__ void g8_put<float>(uint32_t win, int lane, const uint32_t* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts128(win + lane * 128 + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
template <>
__device__ __forceinline__ void g8_put<__nv_bfloat16>(uint32_t win, int lane, const uint32_t* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = ops_bf2(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
    sts128(win + lane * 128 + ((j ^ (lane & 7)) << 4), u[0], u[1], u[2], u[3]);
  }
}

// A window's rows to global memory at any alignment: lane `lane` takes word `lane`
// of each row.  Element i of row r lies at r * 128 + (((chunk of i) ^ (r & 7)) << 4);
// rows come by eights, so r & 7 is known and an address costs one exclusive or.
__device__ __forceinline__ void g8_store_rows(const char* w, float* dst, long long ldc, int rows, int n, int lane,
                                              int accumulate) {
  const char* a = w + (lane & 3) * 4;
  const int q = lane >> 2;
  float* p = dst + lane;
  for (int r0 = 0; r0 < rows; r0 += 8, a += 1024) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const float*>(a + j * 128 + ((q ^ j) << 4));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (lane < n && r0 + j < rows) *p = accumulate ? *p + v[j] : v[j];
      p += ldc;
    }
  }
}
// bf16: words start at even elements, so a row at an odd address has its first
// element apart and words one element on; with an odd ldc that is every other row.
__device__ __forceinline__ void g8_store_rows(const char* w, __nv_bfloat16* dst, long long ldc, int rows, int n,
                                              int lane, int) {
  const int odd0 = (int)((uintptr_t)dst >> 1) & 1, odd1 = odd0 ^ (int)(ldc & 1);
  const char* a = w;
  uint16_t* p = reinterpret_cast<uint16_t*>(dst) + 2 * lane;
  for (int r0 = 0; r0 < rows; r0 += 8, a += 1024) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = 2 * lane + (j & 1 ? odd1 : odd0), y = x < 63 ? x + 1 : 63;
      v[j] = *reinterpret_cast<const uint16_t*>(a + j * 128 + (((x >> 3) ^ j) << 4) + (x & 7) * 2) |
             (uint32_t)*reinterpret_cast<const uint16_t*>(a + j * 128 + (((y >> 3) ^ j) << 4) + (y & 7) * 2) << 16;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int odd = j & 1 ? odd1 : odd0, x = 2 * lane + odd;
      if (r0 + j < rows) {
        if (x + 1 < n && x < 63) *reinterpret_cast<uint32_t*>(p + odd) = v[j];
        else if (x < n) p[odd] = (uint16_t)v[j];
        if (odd && lane == 0) *p = *reinterpret_cast<const uint16_t*>(a + j * 128 + (j << 4));
      }
      p += ldc;
    }
  }
}

// BN: columns of a tile.  BCOL: B has a scale per row (column of C) instead of
// one per 128.  CT: type of C.
template <int BN, bool BCOL, class CT>
__global__ void __launch_bounds__(G8_THREADS, 1) gemm8_k(const __grid_constant__ G8Args g) {
  extern __shared__ __align__(1024) char gen[];
  constexpr int STAGE = G8_A_BYTES + BN * 128;
  constexpr int STAGES = G8_STAGES;
  constexpr int HALF = BN == 64 ? 64 : BN / 2;        // columns per epilogue warp (a window holds 64 of bf16)
  constexpr int EW = 4 * (BN / HALF);                 // epilogue warps
  constexpr int CW = 128 / (int)sizeof(CT);           // columns of a window
  constexpr int ND = BN == 256 ? 1 : 2;               // accumulators (TMEM has 512 columns, scales take 48)
  constexpr int SF = ND * BN;                         // TMEM columns of the scales: slots of 4 (A) + 8 (B)
  static_assert(SF + 12 * G8_SLOTS <= 512, "accumulators and scales exceed TMEM");
  const uint32_t base = smem_u32(gen);
  if (base & 1023) {                                  // swizzled tiles start on 1024-byte boundaries
    if (threadIdx.x == 0 && atomicCAS(g.status, 0, (int)MT_ERR_LAUNCH) == 0) g.status[1] = SITE_TC_ALIGN;
    return;
  }
  volatile int* abort = reinterpret_cast<volatile int*>(gen + G8_ABORT);
  int* offs = reinterpret_cast<int*>(gen + G8_OFFS);
  const uint32_t full = base + G8_BAR, empty = full + 8 * STAGES, tfull = empty + 8 * STAGES, tempty = tfull + 16;
  const uint32_t sready = tempty + 16, sfree = sready + 8 * G8_SLOTS, sabar = sfree + 8 * G8_SLOTS, done = sabar + 8;
  const uint32_t stages = base + G8_DATA;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, EW);
    }
    for (int i = 0; i < G8_SLOTS; ++i) {
      mbar_init(sready + 8 * i, 1);
      mbar_init(sfree + 8 * i, 1);
    }
    mbar_init(sabar, 1);
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + G8_TMEM), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  ops_wait();          // (and no early release: kernels that move in as its CTAs end cost 5 to 15 us)
  // segment starts, kept inside the operands and on block boundaries whatever
  // they hold (a TMA coordinate has to be a multiple of 16)
  if (g.mode != G8_DENSE && tid <= g.nseg) {
    const int lim = ((g.mode == G8_ROWS ? g.M : g.K) + 127) & ~127, v = g.offs[tid] & ~127;
    offs[tid] = v < 0 ? 0 : v > lim ? lim : v;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gen + G8_TMEM);

  const int ntiles = g8_tiles(g, offs), first = g8_first(g, offs) + (int)blockIdx.x;
  // The loading warps need few registers, the storing ones 128 for their part
  // of the tile: the split gives away only what the launch has.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G8_REGS_LOAD));
    if (warp == 0 && lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += gridDim.x) {
        const G8Tile ti = g8_tile<BN>(g, offs, t);
        const int by = (g.mode == G8_ROWS ? ti.seg * g.N : 0) + ti.n0;
        for (int kb = 0; kb < ti.nkb; ++kb, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES && !g8_wait(empty + 8 * s, (it / STAGES - 1) & 1, abort, g.status, SITE_TC_EMPTY)) {
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
        for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i) {
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(full + 8 * (i % STAGES), (i / STAGES) & 1) &&
                 (long long)(globaltimer() - t0) < G8_TIMEOUT_NS) {
          }
        }
    }
    if (warp == 1) {
      // e4m3 x e4m3 with power-of-two scale bytes, both K-major
      const uint32_t idesc = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 4) << 24);
      int nt = 0;                      // sums begun
      uint32_t gi = 0;                 // group of four blocks
      uint32_t s = 0, ph = 0;          // stage and its phase
      const uint64_t ad0 = sdesc(stages, 16, 1024), bd0 = sdesc(stages + G8_A_BYTES, 16, 1024);
      uint64_t ad = ad0, bd = bd0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += gridDim.x) {
        const int nkb = g8_blocks(g, offs, t);
        for (int kc = 0; kc < nkb && ok; kc += G8_CHUNK) {
          const int end = nkb - kc < G8_CHUNK ? nkb : kc + G8_CHUNK;
          const int d = nt % ND;
          if (nt >= ND && !g8_wait_warp(tempty + 8 * d, (nt / ND - 1) & 1, abort, g.status, SITE_TC_ACC_EMPTY)) {
            ok = false;
            break;
          }
          ++nt;
          uint32_t acc = 0;
          for (int kb = kc; kb < end && ok; kb += 4, ++gi) {
            const uint32_t slot = gi % G8_SLOTS, sf = tmem + SF + slot * 12;
            if (!(ok = g8_wait_warp(sready + 8 * slot, (gi / G8_SLOTS) & 1, abort, g.status, SITE_TC_QUEUE))) break;
            const int n = end - kb < 4 ? end - kb : 4;
            uint32_t id = idesc;
            for (int i = 0; i < n; ++i) {
              if (!(ok = g8_wait_warp(full + 8 * s, ph, abort, g.status, SITE_TC_FULL))) break;
              tc_fence_after();
              g8_mma_block(tmem + d * BN, ad, bd, id, sf, sf + 4, acc, empty + 8 * s);
              acc = 1;
              id += (1u << 4) | (1u << 29);          // the next scale byte of each word
              ad += STAGE >> 4;
              bd += STAGE >> 4;
              if (++s == STAGES) {
                s = 0;
                ph ^= 1;
                ad = ad0;
                bd = bd0;
              }
            }
            mma_commit_warp(sfree + 8 * slot);
          }
          if (ok) mma_commit_warp(tfull + 8 * d);
        }
      }
      // every issued product has arrived before the TMEM is freed
      mma_commit_warp(done);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(done, 0) && (long long)(globaltimer() - t0) < G8_TIMEOUT_NS) {
      }
    }
    if (warp >= 2) {
      // Scale bytes of four blocks as one word per row: warp 2 A's rows lane +
      // 32 j, warp 3 B's (or its one or two blocks of 128 rows).  Rows past the edge
      // repeat the last one, bytes past the last block are any: they multiply zeros
      // or nothing.  A
      // group is read while the one before it waits for its place, across tiles
      // too: a read begun when it is due would hold the products up for its trip.
      constexpr int NR = BN > 128 ? 8 : 4;
      const bool isa = warp == 2, words = isa ? g.words_a : g.words_b;
      G8Tile ti;
      ti.nkb = 0;
      int t = first - (int)gridDim.x, kb = -4;
      auto advance = [&]() {
        kb += 4;
        while (kb >= ti.nkb) {
          t += gridDim.x;
          if (t >= ntiles) return false;
          ti = g8_tile<BN>(g, offs, t);
          kb = 0;
        }
        return true;
      };
      // Row starts of the tile, and the words of a group as they were read: they
      // are used a whole group later.
      const uint8_t* p[NR];
      uint32_t lo[NR], hi[NR];
      int sh = 0;
      auto load = [&]() {
        if (kb == 0) {
          const long long seg = g.mode == G8_ROWS ? ti.seg : 0;
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            long long r;
            if (isa) {
              const int m = ti.m0 + 32 * (j & 3) + lane;
              r = (m < g.M ? m : g.M - 1) * g.ldsa;
            } else if (BCOL) {
              const int c = ti.n0 + 32 * j + lane;
              r = (seg * g.N + (c < g.N ? c : g.N - 1)) * g.ldsb;
            } else {
              const int nrb = (g.N + 127) >> 7, b = (ti.n0 >> 7) + (j >> 2);
              r = (seg * nrb + (b < nrb ? b : nrb - 1)) * g.ldsb;
            }
            p[j] = (isa ? g.sa : g.sb) + r + (ti.k0 >> 7);
          }
        }
        const int n = ti.nkb - kb < 4 ? ti.nkb - kb : 4;
        sh = words ? (int)((uintptr_t)(p[0] + kb) & 3) : 0;      // the same in every row
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if (isa ? j > 3 : !BCOL && (j & 3)) continue;
          if (words) {
            // the aligned words that hold the bytes lie in the same row
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p[j] + kb - sh);
            lo[j] = q[0];
            hi[j] = sh + n > 4 ? q[1] : 0;
          } else {
            lo[j] = hi[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) lo[j] |= (uint32_t)p[j][kb + (i < n ? i : n - 1)] << (8 * i);
          }
        }
      };
      bool have = advance();
      if (have) load();
      uint32_t it = 0;
      for (; have; ++it) {
        uint32_t w[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const int k = isa ? j & 3 : BCOL ? j : j & 4;
          w[j] = __funnelshift_r(lo[k], hi[k], 8 * sh);
        }
        have = advance();
        if (have) load();
        // the copy of the group before has read the bytes
        const uint32_t was = (it - 1) % G8_SLOTS, slot = it % G8_SLOTS;
        if (it > 0 && !g8_wait_warp(sready + 8 * was, ((it - 1) / G8_SLOTS) & 1, abort, g.status, SITE_TC_QUEUE)) break;
        const uint32_t dst = base + (isa ? G8_SFA : G8_SFB) + 16 * lane;
        sts128(dst, w[0], w[1], w[2], w[3]);
        if (NR == 8 && !isa) sts128(dst + 512, w[4 % NR], w[5 % NR], w[6 % NR], w[7 % NR]);
        fence_smem_async();
        __syncwarp();
        if (isa) {
          if (lane == 0) mbar_arrive(sabar);
        } else {
          // A's bytes are there, and the products of the slot's last group are done
          if (!g8_wait_warp(sabar, it & 1, abort, g.status, SITE_TC_QUEUE)) break;
          if (it >= G8_SLOTS && !g8_wait_warp(sfree + 8 * slot, (it / G8_SLOTS - 1) & 1, abort, g.status, SITE_TC_DRAIN)) break;
          tc_fence_after();
          const uint32_t c = tmem + SF + slot * 12;
          g8_copy_scales(c, base + G8_SFA);
          g8_copy_scales(c + 4, base + G8_SFB);
          if (BN > 128) g8_copy_scales(c + 8, base + G8_SFB + 512);
          mma_commit_warp(sready + 8 * slot);
        }
      }
      // the last copy has arrived before the TMEM is freed
      if (!isa && it > 0) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(sready + 8 * ((it - 1) % G8_SLOTS), ((it - 1) / G8_SLOTS) & 1) &&
               (long long)(globaltimer() - t0) < G8_TIMEOUT_NS) {
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G8_REGS_EPI));
    const int ew = warp - 4, quad = warp & 3, half = ew >> 2;
    const uint32_t win = stages + STAGES * STAGE + ew * G8_WIN;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + half * HALF;
    int nt = 0;
    bool ok = true;
    for (int t = ew < EW ? first : ntiles; t < ntiles && ok; t += gridDim.x) {
      const G8Tile ti = g8_tile<BN>(g, offs, t);
      const int col = ti.n0 + half * HALF;
      uint32_t acc[HALF];
      for (int kc = 0; kc < ti.nkb; kc += G8_CHUNK, ++nt) {
        const int d = nt % ND;
        ok = g8_wait_warp(tfull + 8 * d, (nt / ND) & 1, abort, g.status, SITE_TC_ACC_FULL);
        if (!ok) break;
        tc_fence_after();
        if (kc == 0) {
#pragma unroll
          for (int c = 0; c < HALF; c += 32) g8_ld32(trow + d * BN + c, acc + c);
#pragma unroll
          for (int c = 0; c < HALF; c += 32) g8_ld_wait(acc + c);
        } else {
#pragma unroll
          for (int c = 0; c < HALF; c += 32) {
            uint32_t v[32];
            g8_ld32(trow + d * BN + c, v);
            g8_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c + i] = __float_as_uint(__uint_as_float(acc[c + i]) + __uint_as_float(v[i]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty + 8 * d);
      }
      if (!ok) break;
      if (ti.nkb == 0) {
        if (g.accumulate) continue;
#pragma unroll
        for (int i = 0; i < HALF; ++i) acc[i] = 0;
      }
      const int z = g.mode == G8_REDUCE ? ti.seg : 0, row0 = ti.m0 + quad * 32;
      if (col >= g.N || row0 >= g.M) continue;
#pragma unroll
      for (int c = 0; c < HALF; c += CW) {
        if (col + c >= g.N) continue;
        if (lane == 0) bulk_wait_read<0>();        // the store before has left the window
        __syncwarp();
        g8_put<CT>(win, lane, acc + c);
        if (g.tma_out) {
          fence_smem_async();
          __syncwarp();
          if (lane == 0) {
            if (sizeof(CT) == 4 && g.accumulate) g8_add_3d(&g.c, win, col + c, row0, z);
            else g8_store_3d(&g.c, win, col + c, row0, z);
            bulk_commit();
          }
        } else {
          // rows of any alignment: the window is read back eight rows at a time and
          // leaves in 4-byte words
          __syncwarp();
          const int rows = g.M - row0 < 32 ? g.M - row0 : 32;
          g8_store_rows(gen + (win - base), reinterpret_cast<CT*>(g.out) + ((long long)z * g.M + row0) * g.ldc + col + c,
                        g.ldc, rows, g.N - col - c, lane, g.accumulate);
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
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
  if (tiles > 0x3fffffff) return MT_ERR_UNSUPPORTED;
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
  g.words_a = ops_aligned(a->scales, 4) && a->lds % 4 == 0;
  g.words_b = ops_aligned(b->scales, 4) && b->lds % 4 == 0;
  const int which = (bn == 256 ? 0 : bn == 128 ? 4 : 8) + (bcol ? 2 : 0) + (f32 ? 1 : 0);
  G8Kernel k = bn == 256 ? kernel_of<256>(bcol, f32) : bn == 128 ? kernel_of<128>(bcol, f32) : kernel_of<64>(bcol, f32);
  const int smem = g8_smem(bn);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_dev[dev].prepared[which]) {
      cudaFuncAttributes fa;
      // the register split waits for registers that a launch with fewer never frees
      if (cudaFuncGetAttributes(&fa, k) != cudaSuccess || fa.numRegs < G8_REGS ||
          cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return MT_ERR_LAUNCH;
      }
      g_dev[dev].prepared[which] = true;
    }
  }
  return ops_launch(k, (unsigned)(tiles < sms ? tiles : sms), G8_THREADS, smem, st, 1, g);
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
