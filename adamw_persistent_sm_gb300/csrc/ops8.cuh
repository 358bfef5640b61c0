// ops8.cuh - what the stand-alone expert operators share: 8-element row
// accesses, the 8-bit quantiser's arithmetic and the host-side checks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_train.h"

#define OPS_MAX_ROWS (1LL << 30)

// ---------------------------------------------------------------------------
// device
// ---------------------------------------------------------------------------
// First thing in every kernel: let the next one of the stream be launched while
// this one runs, and wait for the one before to be done with its memory (both
// without effect where the launch does not ask for it, see ops_launch).  What a
// kernel reads may thus be written while it is already resident: plain loads, no
// read-only ones.
__device__ __forceinline__ void ops_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void ops_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ops_wait();
}

// n_rows of the C ABI: rows below *p (clamped), or all of them
__device__ __forceinline__ int ops_row_limit(const int* p, int rows) {
  if (!p) return rows;
  const int v = *p;
  return v < 0 ? 0 : v < rows ? v : rows;
}

// Elements c..c+7 of a row, zeros from column n on.  VEC 0: any alignment (S: the
// step between a lane's elements; 32 makes neighbouring lanes take neighbours, where
// it does not matter which lane has which); 1: row
// start and c are 16-byte aligned; 2: and every lane's eight lie inside the row
// and (fp32) on 32-byte boundaries, which the launch knows from the sizes: no test
// per access, the loads of a loop stay together, and fp32 lanes move whole sectors
// (two 16-byte halves each left every sector written twice: 27 against 20 us for
// 4096 x 8 rows of 768).
template <int VEC, int S = 1>
__device__ __forceinline__ void ops_ld8(const float* p, int c, int n, float* v) {
  if constexpr (VEC == 2) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p + c));
    return;
  }
  if (VEC == 2 || (VEC && c + 8 <= n)) {
    const float4 a = *reinterpret_cast<const float4*>(p + c), b = *reinterpret_cast<const float4*>(p + c + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
  if constexpr (VEC != 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i * (VEC ? 1 : S) < n ? p[c + i * (VEC ? 1 : S)] : 0.f;
  }
}
__device__ __forceinline__ float ops_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float ops_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
template <int VEC, int S = 1>
__device__ __forceinline__ void ops_ld8(const __nv_bfloat16* p, int c, int n, float* v) {
  if (VEC == 2 || (VEC && c + 8 <= n)) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + c);
    v[0] = ops_lo(u.x); v[1] = ops_hi(u.x); v[2] = ops_lo(u.y); v[3] = ops_hi(u.y);
    v[4] = ops_lo(u.z); v[5] = ops_hi(u.z); v[6] = ops_lo(u.w); v[7] = ops_hi(u.w);
    return;
  }
  if constexpr (VEC != 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i * (VEC ? 1 : S) < n ? __bfloat162float(p[c + i * (VEC ? 1 : S)]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t ops_bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int VEC, int S = 1>
__device__ __forceinline__ void ops_st8(float* p, int c, int n, const float* v) {
  if constexpr (VEC == 2) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + c), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
    return;
  }
  if (VEC == 2 || (VEC && c + 8 <= n)) {
    *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  if constexpr (VEC != 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * (VEC ? 1 : S) < n) p[c + i * (VEC ? 1 : S)] = v[i];
  }
}
template <int VEC, int S = 1>
__device__ __forceinline__ void ops_st8(__nv_bfloat16* p, int c, int n, const float* v) {
  if (VEC == 2 || (VEC && c + 8 <= n)) {
    *reinterpret_cast<uint4*>(p + c) =
        make_uint4(ops_bf2(v[0], v[1]), ops_bf2(v[2], v[3]), ops_bf2(v[4], v[5]), ops_bf2(v[6], v[7]));
    return;
  }
  if constexpr (VEC != 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * (VEC ? 1 : S) < n) p[c + i * (VEC ? 1 : S)] = __float2bfloat16_rn(v[i]);
  }
}
// Eight codes; `v8`: the address is 8-byte aligned.
template <int VEC>
__device__ __forceinline__ void ops_st_codes(uint8_t* p, int c, int n, uint2 q, bool v8) {
  if (VEC == 2 || (v8 && c + 8 <= n)) {
    *reinterpret_cast<uint2*>(p + c) = q;
    return;
  }
  if constexpr (VEC != 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}
template <int VEC>
__device__ __forceinline__ uint2 ops_ld_codes(const uint8_t* p, int c, int n, bool v8) {
  uint2 q = make_uint2(0, 0);
  if (VEC == 2 || (v8 && c + 8 <= n)) {
    q = *reinterpret_cast<const uint2*>(p + c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = c + i < n ? p[c + i] : 0;
      if (i < 4) q.x |= b << (8 * i);
      else q.y |= b << (8 * (i - 4));
    }
  }
  return q;
}

// Infinite and NaN elements become NaN (which the conversion turns into the
// e4m3 NaN).
__device__ __forceinline__ float ops_finite(float x) {
  return fabsf(x) <= 3.402823466e38f ? x : __int_as_float(0x7fffffff);
}
// The block's scale from the bits of its largest magnitude 1.f * 2^x: e, the least
// with amax <= 448 * 2^e = 1.75 * 2^(e + 8), is x - 8, one more where 1.f > 1.75 -
// where adding 0x1fffff carries into the exponent.  At least -126, 0 for amax = 0.
// `byte` e + 127; the result 2^-e.
__device__ __forceinline__ float ops_scale(uint32_t top, uint32_t* byte) {
  uint32_t x = (top + 0x1fffffu) >> 23;
  x = top ? max(x, 9u) : 135u;
  *byte = x - 8;
  return __uint_as_float((262u - x) << 23);
}
// What a scale byte stands for, as the products read it: 2^(byte - 127), subnormal
// for 0, and NaN for 255 - the two whose bits need more than the exponent's place.
__device__ __forceinline__ float ops_byte_scale(uint32_t byte) {
  return __uint_as_float(byte << 23 | (((byte + 1) & 0xff) <= 1 ? 0x400000u : 0u));
}
// four e4m3 codes of v * s (round to nearest even; |v * s| <= 448 or NaN); the
// products two at a time (one issue slot for both)
__device__ __forceinline__ uint32_t ops_codes4(float v0, float v1, float v2, float v3, float s) {
  uint32_t q;
  asm("{\n\t.reg .b64 a, b, s;\n\t.reg .f32 x, y, z, w;\n\t.reg .b16 lo, hi;\n\t"
      "mov.b64 s, {%5, %5};\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "mul.rn.f32x2 a, a, s;\n\t"
      "mul.rn.f32x2 b, b, s;\n\t"
      "mov.b64 {x, y}, a;\n\t"
      "mov.b64 {z, w}, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, y, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, w, z;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(q)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(s));
  return q;
}
__device__ __forceinline__ uint32_t ops_codes4(const float* v, float s) { return ops_codes4(v[0], v[1], v[2], v[3], s); }
__device__ __forceinline__ uint2 ops_codes8(const float* v, float s) {
  return make_uint2(ops_codes4(v, s), ops_codes4(v + 4, s));
}
// values of eight codes, times s
__device__ __forceinline__ void ops_values8(uint2 q, float s, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t h = (uint16_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1)));
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&f));
    v[2 * i] = t.x * s;
    v[2 * i + 1] = t.y * s;
  }
}
// ---------------------------------------------------------------------------
// Eight elements of a row as they lie in memory.  Magnitudes are compared as
// integers - the bits of |x|, whose order is the values' and which put
// infinities and NaN on top - so that a block's maximum also tells whether
// every element is finite: the rare block with others is looked at again, and
// the usual one pays nothing per element for the question.
// ---------------------------------------------------------------------------
#define OPS_INF 0x7f800000u
__device__ __forceinline__ uint32_t ops_max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// largest magnitude of three, NaN if any is
__device__ __forceinline__ float ops_max3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  template <int VEC, int S = 1>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int c, int n) {
    if (VEC == 2 || (VEC && c + 8 <= n)) {
      u = *reinterpret_cast<const uint4*>(p + c);
      return;
    }
    if constexpr (VEC != 2) {
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = c + i * (VEC ? 1 : S) < n ? reinterpret_cast<const uint16_t*>(p)[c + i * (VEC ? 1 : S)] : 0;
      u = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
  }
  template <int VEC, int S = 1>
  __device__ __forceinline__ void store(__nv_bfloat16* p, int c, int n) const {
    if (VEC == 2 || (VEC && c + 8 <= n)) {
      *reinterpret_cast<uint4*>(p + c) = u;
      return;
    }
    if constexpr (VEC != 2) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i * (VEC ? 1 : S) < n) reinterpret_cast<uint16_t*>(p)[c + i * (VEC ? 1 : S)] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  }
  // bits (fp32) of the largest magnitude
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = ops_max_u16x2(ops_max_u16x2(u.x & m, u.y & m), ops_max_u16x2(u.z & m, u.w & m));
    return max(a << 16, a & 0xffff0000u);
  }
  __device__ __forceinline__ void values(float* v) const {
    v[0] = ops_lo(u.x); v[1] = ops_hi(u.x); v[2] = ops_lo(u.y); v[3] = ops_hi(u.y);
    v[4] = ops_lo(u.z); v[5] = ops_hi(u.z); v[6] = ops_lo(u.w); v[7] = ops_hi(u.w);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  template <int VEC, int S = 1>
  __device__ __forceinline__ void load(const float* p, int c, int n) {
    float v[8];
    ops_ld8<VEC, S>(p, c, n, v);
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  template <int VEC, int S = 1>
  __device__ __forceinline__ void store(float* p, int c, int n) const {
    float v[8];
    values(v);
    ops_st8<VEC, S>(p, c, n, v);
  }
  __device__ __forceinline__ uint32_t top() const {
    const float m = ops_max3(ops_max3(a.x, a.y, a.z), ops_max3(a.w, b.x, b.y), b.z);
    return __float_as_uint(ops_max3(m, b.w, b.w));
  }
  __device__ __forceinline__ void values(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
// the same of values in registers
__device__ __forceinline__ uint32_t ops_top8(const float* v) {
  const float m = ops_max3(ops_max3(v[0], v[1], v[2]), ops_max3(v[3], v[4], v[5]), v[6]);
  return __float_as_uint(ops_max3(m, v[7], v[7]));
}
// maximum over the 16 lanes that hold one block of 128
__device__ __forceinline__ uint32_t ops_max16(uint32_t a) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}
// Codes of eight elements v of a block whose largest magnitude (over 16 lanes)
// has the bits `top`, and the block's scale byte.  The whole warp calls it.
__device__ __forceinline__ uint2 ops_quantise(float* v, uint32_t top, uint32_t* byte) {
  if (__any_sync(0xffffffffu, top >= OPS_INF)) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = ops_finite(v[i]);
      if (v[i] == v[i]) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    top = ops_max16(m);
  }
  return ops_codes8(v, ops_scale(top, byte));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static inline bool ops_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
static inline int ops_size(int dtype) { return dtype == MT_DT_FP32 ? 4 : 2; }
static inline bool ops_dtype_ok(int dtype) { return dtype == MT_DT_FP32 || dtype == MT_DT_BF16; }
// a matrix of the caller: non-null, aligned to its element, rows at least as long as they are used
static inline bool ops_mat_ok(const void* p, int dtype, int64_t ld, int64_t cols) {
  return p && ops_aligned(p, ops_size(dtype)) && ld >= cols && ld <= (1LL << 40);
}
// access to every row of a matrix: 0 by element, 1 by 16 bytes, 2 by the eight
// elements of a lane (16 bytes of bf16, 32 of fp32)
static inline int ops_vec(const void* p, int dtype, int64_t ld) {
  const int64_t b = ld * ops_size(dtype);
  const int whole = 8 * ops_size(dtype);
  return ops_aligned(p, whole) && b % whole == 0 ? 2 : ops_aligned(p, 16) && b % 16 == 0 ? 1 : 0;
}
static inline int ops_least(int a, int b) { return a < b ? a : b; }
// the mode of ops_ld8 for rows of `width` columns taken `chunk` at a time
static inline int ops_mode(int vec, int64_t width, int chunk) { return vec == 2 && width % chunk ? 1 : vec; }
static inline int64_t ops_blocks(const mt_mat8* m) {
  return m->halves ? 2 * ((m->cols / 2 + 127) / 128) : (m->cols + 127) / 128;
}
static inline bool ops_mat8_ok(const mt_mat8* m) {
  if (!m || !m->codes || !m->scales || m->reserved0) return false;
  if (m->rows < 0 || m->cols < 1 || m->batch < 1 || m->cols > OPS_MAX_ROWS) return false;
  if (m->rows > OPS_MAX_ROWS || m->rows * m->batch > OPS_MAX_ROWS) return false;
  if (m->block_rows != 1 && m->block_rows != 128) return false;
  if (m->halves != 0 && (m->halves != 1 || m->block_rows != 1 || m->cols % 2)) return false;
  if (!ops_aligned(m->codes, 16) || m->ld % 16 || m->ld < m->cols || m->ld > (1LL << 40)) return false;
  return m->lds >= ops_blocks(m) && m->lds <= (1LL << 40);
}
// A launch that may become resident while the kernel before it in the stream
// drains (a chain of moves loses 3 to 5 us per boundary otherwise); `cluster` CTAs
// per cluster.
template <class... P, class... A>
static int ops_launch(void (*k)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, unsigned cluster,
                      A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, k, (P)args...) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  return MT_OK;
}
