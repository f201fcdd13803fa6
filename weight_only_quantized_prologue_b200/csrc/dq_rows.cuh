// dq_rows.cuh -- the row operators around the block-scaled FP8 products: the
// RMS norm with the residual's addition, the gated SiLU and the activation
// quantizer.  Inputs bf16, fp16 or fp32; outputs in one of those types, as
// e4m3 codes with an fp32 scale per 128 elements of a row, or as e4m3 codes
// under one given scale.  All arithmetic is fp32.
//
// All of them are bound by HBM: each input is read once and each output
// written once.  A thread works on vectors of 8 consecutive elements (one
// 16-byte load in 16 bits, one 8-byte store of codes), and 16 neighbouring
// lanes hold one block of 128, so a block's maximum is four shuffles.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dq_common.cuh"

namespace dq {

enum RowType { ROW_BF16 = 0, ROW_FP16 = 1, ROW_FP32 = 2 };
enum RowOut { OUT_BF16 = 0, OUT_FP16 = 1, OUT_FP32 = 2, OUT_BLOCK = 3, OUT_STATIC = 4 };

constexpr int QBLOCK = 128;   // elements of a row per scale

struct RowArgs {
  const void* x;          // [M, K] (gate: [M, 2K], the gate's half first), rows ldx elements apart
  long long ldx;
  const void* res;        // rmsnorm: residual [M, K] or null
  void* res_out;          //   x + residual, rounded to the input type (null without a residual)
  const void* w;          //   weight [K] or null (ones)
  int w_type;             //   its RowType
  float eps;
  int M, K;
  void* out;              // [M, K]
  float* scales;          // OUT_BLOCK: [M, ceil(K / 128)]
  float s_out, r_out;     // OUT_STATIC: the scale and f32(1 / s_out)
};

// ---------------------------------------------------------------------------
// 8 consecutive elements <-> fp32.  AL: rows are 16-byte aligned and K a
// multiple of 8, so a vector is whole; else n of its elements exist (n <= 0:
// none) and they are taken one by one.  Missing elements read as 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (sizeof(T) == 2) {
    const T u = from_f32<T>(a), v = from_f32<T>(b);
    return (uint32_t)*reinterpret_cast<const uint16_t*>(&u) | ((uint32_t)*reinterpret_cast<const uint16_t*>(&v) << 16);
  } else {
    return 0u;
  }
}

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __half) {
  const __half2 h = *reinterpret_cast<const __half2*>(&w);
  a = __low2float(h);
  b = __high2float(h);
}

template <bool AL, typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if constexpr (AL) {
    if (n > 0) {
      if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        unpack2(u.x, v[0], v[1], T());
        unpack2(u.y, v[2], v[3], T());
        unpack2(u.z, v[4], v[5], T());
        unpack2(u.w, v[6], v[7], T());
      } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

template <bool AL, typename T>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
  if constexpr (AL) {
    if (n > 0) {
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                                  pack2<T>(v[6], v[7]));
      } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

template <bool AL>
__device__ __forceinline__ void load8_typed(const void* p, int type, long long at, int n, float (&v)[8]) {
  if (type == ROW_BF16)
    load8<AL>(static_cast<const __nv_bfloat16*>(p) + at, n, v);
  else if (type == ROW_FP16)
    load8<AL>(static_cast<const __half*>(p) + at, n, v);
  else
    load8<AL>(static_cast<const float*>(p) + at, n, v);
}

// ---------------------------------------------------------------------------
// quantization to e4m3
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The scale of a block, s = f32(amax / 448), and r = f32(1 / s) (1 for s = 0),
// from the bits of amax.  Straight-line: both quotients by Markstein's
// correction steps (see e4m3_quotient), r from the hardware's reciprocal
// (within 2^-23) by one step, which gives the correctly rounded value unless
// s has the largest significand.  `fast` says that s and r are what they
// should be and that r is a normal number: amax is 0, or from 2^-87 to the
// largest finite value, and s has another significand.  The division's own
// code has branches for special operands (zero among them, the commonest
// block of all) that keep several blocks from being worked on at once.
struct BlockScale {
  float s, r;
  bool fast;
};
__device__ __forceinline__ BlockScale block_scale_of(uint32_t amax_bits) {
  constexpr float r448 = 1.f / 448.f;
  const float a = __uint_as_float(amax_bits);
  const float q0 = __fmul_rn(a, r448);
  BlockScale b;
  b.s = __fmaf_rn(__fmaf_rn(-q0, 448.f, a), r448, q0);
  const float d = amax_bits == 0u ? 1.f : b.s;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
  b.r = __fmaf_rn(y, __fmaf_rn(-d, y, 1.f), y);
  b.fast = amax_bits == 0u || (amax_bits - 0x14000000u < 0x7F800000u - 0x14000000u &&
                               (__float_as_uint(b.s) & 0x7FFFFFu) != 0x7FFFFFu);
  return b;
}

// f32(v / s), correctly rounded where the e4m3 code depends on it, without
// the range test of e4m3_quotient: for r = f32(1 / s) normal and |v / s| not
// above 2^9, the correction leaves every quotient below 2^-12 there (where
// each code is 0) and cannot overflow.  The sign is v's, of a zero too.
__device__ __forceinline__ float block_quotient(float v, float s, float r) {
  const float q0 = __fmul_rn(v, r);
  const float q = __fmaf_rn(__fmaf_rn(-q0, s, v), r, q0);
  return __uint_as_float((__float_as_uint(q) & 0x7FFFFFFFu) | (__float_as_uint(v) & 0x80000000u));
}

// The 8 codes of v under the scale s: e4m3(f32(v / s)), 0 where s is 0; for
// blocks whose scale is `fast` ...
__device__ __forceinline__ uint2 codes8_fast(const float (&v)[8], float s, float r) {
  const uint32_t lo = e4m3x2(block_quotient(v[0], s, r), block_quotient(v[1], s, r)) |
                      (e4m3x2(block_quotient(v[2], s, r), block_quotient(v[3], s, r)) << 16);
  const uint32_t hi = e4m3x2(block_quotient(v[4], s, r), block_quotient(v[5], s, r)) |
                      (e4m3x2(block_quotient(v[6], s, r), block_quotient(v[7], s, r)) << 16);
  return s == 0.f ? make_uint2(0u, 0u) : make_uint2(lo, hi);
}
// ... and for any scale, by the division (a NaN makes every code of its block
// NaN; in a block with an infinity the finite elements' codes are 0)
static __device__ __noinline__ uint2 codes8_any(const float (&v)[8], float s) {
  if (s == 0.f) return make_uint2(0u, 0u);
  const uint32_t lo = e4m3x2(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s)) | (e4m3x2(__fdiv_rn(v[2], s), __fdiv_rn(v[3], s)) << 16);
  const uint32_t hi = e4m3x2(__fdiv_rn(v[4], s), __fdiv_rn(v[5], s)) | (e4m3x2(__fdiv_rn(v[6], s), __fdiv_rn(v[7], s)) << 16);
  return make_uint2(lo, hi);
}

// Bits of the largest magnitude of the 128 elements that 16 neighbouring lanes
// hold.  The bits' order is the values', with NaN above infinity, so a NaN
// makes the scale NaN.  The whole warp calls this.
__device__ __forceinline__ uint32_t block_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// scale and codes of a warp's two blocks (the whole warp calls this)
__device__ __forceinline__ uint2 quantize_block(const float (&v)[8], float* s) {
  const uint32_t m = block_amax(v);
  const BlockScale b = block_scale_of(m);
  if (__all_sync(0xFFFFFFFFu, b.fast)) {
    *s = b.s;
    return codes8_fast(v, b.s, b.r);
  }
  *s = __fdiv_rn(__uint_as_float(m), 448.f);
  return codes8_any(v, *s);
}

template <bool AL>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
  if constexpr (AL) {
    if (n > 0) *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// Vector `vec` (8 elements) of row `row`, n of which exist, to the output.
// The whole warp calls this, its lanes holding consecutive vectors from a
// multiple of 32 on.
template <int OUT, bool AL>
__device__ __forceinline__ void emit8(const RowArgs& a, int row, int vec, int n, const float (&v)[8]) {
  const long long at = (long long)row * a.K + vec * 8;
  if constexpr (OUT == OUT_BLOCK) {
    float s;
    const uint2 c = quantize_block(v, &s);
    if (n > 0) {
      if ((vec & 15) == 0) a.scales[(long long)row * ((a.K + QBLOCK - 1) / QBLOCK) + (vec >> 4)] = s;
      store_codes<AL>(static_cast<uint8_t*>(a.out) + at, n, c);
    }
  } else if constexpr (OUT == OUT_STATIC) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[h] |= (uint32_t)act_code_r(v[4 * h + i], a.s_out, a.r_out) << (8 * i);
    }
    store_codes<AL>(static_cast<uint8_t*>(a.out) + at, n, make_uint2(w[0], w[1]));
  } else if constexpr (OUT == OUT_BF16) {
    store8<AL>(static_cast<__nv_bfloat16*>(a.out) + at, n, v);
  } else if constexpr (OUT == OUT_FP16) {
    store8<AL>(static_cast<__half*>(a.out) + at, n, v);
  } else {
    store8<AL>(static_cast<float*>(a.out) + at, n, v);
  }
}

// ---------------------------------------------------------------------------
// RMS norm:  r = x + residual,  y = r * w / sqrt(mean(r^2) + eps).
// The sum r is kept in fp32 for the norm (only the residual that is stored is
// rounded), so the output carries one rounding.  blockDim.x threads hold a
// row (NV vectors each, read once) and blockDim.y rows share a CTA; NV = 0
// reads the row twice, for rows that do not fit in registers.
// residual_out may be the residual or x itself: every element is read by the
// thread that writes it, before it is written.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    float* p = part + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; ++i) v += p[i];
  }
  return v;
}

template <typename T, int NV, int OUT, bool AL>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const RowArgs a) {
  __shared__ float part[16];
  pdl_launch_dependents();
  pdl_wait();   // x, the residual and the weight may be the previous grid's output
  const int row_raw = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row_raw < a.M;
  const int row = live ? row_raw : 0;
  const int K = a.K;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.ldx;
  const T* res = a.res ? static_cast<const T*>(a.res) + (long long)row * K : nullptr;
  T* res_out = a.res ? static_cast<T*>(a.res_out) + (long long)row * K : nullptr;
  const auto load = [&](int vec, int n, float (&r)[8]) {
    load8<AL>(x + vec * 8, n, r);
    if (res) {
      float b[8];
      load8<AL>(res + vec * 8, n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] += b[i];
    }
  };
  const auto finish = [&](int vec, int n, float rs, float (&r)[8]) {
    float w[8];
    if (a.w) {
      load8_typed<AL>(a.w, a.w_type, vec * 8, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = r[i] * rs * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] *= rs;
    }
    emit8<OUT, AL>(a, row, vec, n, r);
  };
  float sum = 0.f;
  if constexpr (NV > 0) {
    float r[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      const int n = live ? K - vec * 8 : 0;
      load(vec, n, r[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      const int n = live ? K - vec * 8 : 0;
      if (res_out) store8<AL>(res_out + vec * 8, n, r[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(r[i][j], r[i][j], sum);
    }
    const float rs = rsqrtf(row_sum(sum, part) / (float)K + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      finish(vec, live ? K - vec * 8 : 0, rs, r[i]);
    }
  } else {
    const int steps = (K + 8 * (int)blockDim.x - 1) / (8 * (int)blockDim.x);
    float r[8];
    for (int i = 0; i < steps; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      load(vec, live ? K - vec * 8 : 0, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(r[j], r[j], sum);
    }
    const float rs = rsqrtf(row_sum(sum, part) / (float)K + a.eps);
    for (int i = 0; i < steps; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      const int n = live ? K - vec * 8 : 0;
      load(vec, n, r);
      if (res_out) store8<AL>(res_out + vec * 8, n, r);
      finish(vec, n, rs, r);
    }
  }
}

// ---------------------------------------------------------------------------
// gated SiLU  y = g / (1 + e^-g) * u,  and (GATE = false) the plain copy that
// the activation quantizer is.  One vector a thread; `chunks` CTAs a row.
// ---------------------------------------------------------------------------
// FAST (outputs of 16 or 8 bits): the hardware's exponential and reciprocal.
// Their error, about 2^-22 plus 2^-24 per unit of |g|, stays far below half a
// step of the output wherever the result is not itself vanishing.
template <bool FAST>
__device__ __forceinline__ float silu(float g) {
  if constexpr (FAST) return __fdividef(g, 1.f + __expf(-g));
  return g / (1.f + expf(-g));
}

template <typename T, bool GATE, int OUT, bool AL>
__global__ void __launch_bounds__(256) rows_kernel(const RowArgs a, int chunks) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x / chunks;
  const int vec = (blockIdx.x - row * chunks) * 256 + threadIdx.x;
  const int n = a.K - vec * 8;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.ldx;
  float v[8];
  load8<AL>(x + vec * 8, n, v);
  if constexpr (GATE) {
    float u[8];
    load8<AL>(x + a.K + vec * 8, n, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu<OUT != OUT_FP32>(v[i]) * u[i];
  }
  emit8<OUT, AL>(a, row, vec, n, v);
}

}  // namespace dq
