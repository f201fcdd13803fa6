// dq_rows.cuh -- the row operators around the block-scaled FP8 products: the
// RMS norm with the residual's addition, the gated SiLU and the activation
// quantizer.  Inputs bf16, fp16 or fp32; outputs in one of those types, as
// e4m3 codes with an fp32 scale per 128 elements of a row, or as e4m3 codes
// under one given scale.  All arithmetic is fp32.
//
// All of them read each input once and write each output once.  At the rate of
// HBM that leaves about 27 instructions per element of a gated SiLU, so the
// kernels are written for few of them: a thread works on vectors of 16
// consecutive elements (one 32-byte load in 16 bits, one 16-byte store of
// codes), 8 neighbouring lanes hold one block of 128, and what a block costs
// (three shuffles, its scale and reciprocal) is shared by 16 elements a lane.
// With 8 elements a lane the quantizer took 20 instructions an element and
// was bound by their issue (67 to 81 % of the slots, 45 to 70 % of HBM).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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
  long long x_bytes, row_bytes;   // extents of x (gaps between its rows included) and of the residual
  const void* w;          //   weight [K] or null (ones)
  int w_type;             //   its RowType
  float eps;
  int M, K;
  void* out;              // [M, K]
  float* scales;          // OUT_BLOCK: [M, ceil(K / 128)]
  float s_out, r_out;     // OUT_STATIC: the scale and f32(1 / s_out)
};

// ---------------------------------------------------------------------------
// 16 consecutive elements <-> fp32, n of which exist (n <= 0: none); missing
// ones read as 0.  AL = 2: rows are 32-byte aligned and K is a multiple of 16,
// so a vector is whole; 1: 16-byte aligned and a multiple of 8, so each half
// is; 0: rows start anywhere.  A vector of those is read in the aligned
// 16-byte pieces that it touches and shifted into place, and written in
// aligned pieces that neighbouring lanes put together (element by element,
// a norm of 8192 x 4099 in bf16 took 283 us, now 88, a gated SiLU of 4096 x 5003
// 128 us, now 23).  Only pieces that lie within
// the tensor are touched; at its ends it is elements.
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
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Two fp32 values side by side: one instruction works on both.  The kernels
// hold their 16 elements as 8 such pairs.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo(F2 x) { return __uint_as_float((uint32_t)x.v); }
__device__ __forceinline__ float hi(F2 x) { return __uint_as_float((uint32_t)(x.v >> 32)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
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

// 32 bytes in one instruction (sm_100), in program order with the stores
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// N words from byte `off` (0 to 15, a multiple of SIZE) of t on.  `off` is the
// same for a whole warp: a branch on its words costs less than selects (about
// 11 instructions against 27 for 8 words).
template <int N, int SIZE>
__device__ __forceinline__ void shift_words(const uint32_t (&t)[N + 4], uint32_t off, uint32_t (&w)[N]) {
  const auto from = [&](auto words) {
    constexpr int D = decltype(words)::value;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = SIZE == 4 ? t[i + D] : __funnelshift_r(t[i + D], t[i + D + 1], (off & 3) * 8);
  };
  if (off < 8) {
    if (off < 4) from(std::integral_constant<int, 0>());
    else from(std::integral_constant<int, 1>());
  } else {
    if (off < 12) from(std::integral_constant<int, 2>());
    else from(std::integral_constant<int, 3>());
  }
}

// a vector as it lies in memory
template <int AL, typename T>
struct Raw16 {
  static constexpr int PACKED = 4 * sizeof(T);               // words of 16 elements
  static constexpr int WORDS = AL == 0 ? PACKED + 4 : PACKED;
  uint32_t w[WORDS];
  uint32_t off;   // AL = 0: bytes of w before the vector
  int left;       //         elements that exist
  // begin, bytes: the tensor that p points into
  __device__ __forceinline__ void load(const T* p, int n, const void* begin, long long bytes) {
    if constexpr (AL == 0) {
      left = n;
      const uintptr_t at = reinterpret_cast<uintptr_t>(p), piece = at & ~uintptr_t(15), lo_end = reinterpret_cast<uintptr_t>(begin);
      off = (uint32_t)(at & 15);
      if (n > 0 && piece >= lo_end && piece + 4 * WORDS <= lo_end + bytes) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
          const uint4 u = reinterpret_cast<const uint4*>(piece)[i / 4];
          w[i] = u.x;
          w[i + 1] = u.y;
          w[i + 2] = u.z;
          w[i + 3] = u.w;
        }
      } else {
        if (n > 0) off = 0;   // (lanes past the row's end keep the warp's)
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i < n) {
            if constexpr (sizeof(T) == 4) w[i] = bits(p[i]);
            else w[i / 2] |= bits(p[i]) << (16 * (i & 1));
          }
        }
      }
    } else if constexpr (AL == 2) {
      if (n > 0) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 8) ld32(reinterpret_cast<const uint32_t*>(p) + i, *reinterpret_cast<uint32_t(*)[8]>(w + i));
      } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; i += 4) {
        const uint4 u = (i < WORDS / 2 ? n > 0 : n > 8) ? reinterpret_cast<const uint4*>(p)[i / 4] : make_uint4(0u, 0u, 0u, 0u);
        w[i] = u.x;
        w[i + 1] = u.y;
        w[i + 2] = u.z;
        w[i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void values(F2 (&v)[8]) const {
    uint32_t t[PACKED];
    words(t);
    unpack(t, v);
  }
  // the vector's words, those that do not exist as 0 ...
  __device__ __forceinline__ void words(uint32_t (&t)[PACKED]) const {
    if constexpr (AL == 0) {
      shift_words<PACKED, sizeof(T)>(w, off, t);
      if (left < 16) {
#pragma unroll
        for (int i = 0; i < PACKED; ++i) {
          if constexpr (sizeof(T) == 4) t[i] = i < left ? t[i] : 0u;
          else t[i] = 2 * i + 1 < left ? t[i] : 2 * i < left ? t[i] & 0xFFFFu : 0u;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < PACKED; ++i) t[i] = w[i];
    }
  }
  // ... and as numbers
  static __device__ __forceinline__ void unpack(const uint32_t (&t)[PACKED], F2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      if constexpr (sizeof(T) == 4) {
        a = __uint_as_float(t[2 * i]);
        b = __uint_as_float(t[2 * i + 1]);
      } else {
        unpack2(t[i], a, b, T());
      }
      v[i] = f2(a, b);
    }
  }
  static __device__ __forceinline__ uint32_t bits(T v) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(&v);
    else return *reinterpret_cast<const uint16_t*>(&v);
  }
};

template <int AL, typename T>
__device__ __forceinline__ void load16(const T* p, int n, const void* begin, long long bytes, F2 (&v)[8]) {
  Raw16<AL, T> raw;
  raw.load(p, n, begin, bytes);
  raw.values(v);
}

// AL = 0: the 16 elements of SIZE bytes that each lane of a warp holds as W
// words, n of which exist, to its place p (lanes 4 W bytes apart, full ones
// first).  Piece j, the 16 bytes at p - off + 16 j, begins with the last `off`
// bytes of the lane before (j = 0) or of the words before; a lane stores those
// of its pieces that are whole.  The first lane's first piece lacks its start
// and the last lane's last piece its end: they go in powers of two.  (One by
// one, those elements were most of the instructions.)  The whole warp calls this.
template <int W, int SIZE>
__device__ __forceinline__ void store_unaligned(void* p, int n, const uint32_t (&w)[W]) {
  const int lane = threadIdx.x & 31;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  const int bytes = (n < 0 ? 0 : n > 16 ? 16 : n) * SIZE;
  const int next = __shfl_down_sync(0xFFFFFFFFu, bytes, 1);
  uint8_t* piece = static_cast<uint8_t*>(p) - off;
  uint32_t t[W + 8], c[W + 4];   // the last lane's end, this one's words, and their pieces
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __shfl_up_sync(0xFFFFFFFFu, w[W - 4 + i], 1);
    t[W + 4 + i] = 0u;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) t[4 + i] = w[i];
  if (off == 0) {
#pragma unroll
    for (int i = 0; i < W + 4; ++i) c[i] = t[4 + i];
  } else {
    shift_words<W + 4, SIZE>(t, 16 - off, c);
  }
  const bool cut = lane == 0 && off;   // piece 0 lacks its start
  const int end = (int)off + bytes;    // bytes of the pieces that exist
  if (cut && end < 16) {   // and its end
#pragma unroll
    for (int i = 0; i < 16 / SIZE; ++i) {
      if (i * SIZE < bytes) {
        if constexpr (SIZE == 4) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + 4 * i) = w[i];
        else if constexpr (SIZE == 2) *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p) + 2 * i) = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        else static_cast<uint8_t*>(p)[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
      }
    }
  } else if (bytes > 0) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j)
      if (16 * (j + 1) <= end && !(j == 0 && cut))
        *reinterpret_cast<uint4*>(piece + 16 * j) = make_uint4(c[4 * j], c[4 * j + 1], c[4 * j + 2], c[4 * j + 3]);
    if (cut) {   // bytes off to 15, from their end on
      const uint32_t h = 16 - off;
      if (h & 8) *reinterpret_cast<uint2*>(piece + 8) = make_uint2(c[2], c[3]);
      if (h & 4) *reinterpret_cast<uint32_t*>(piece + (h & 8 ? 4 : 12)) = h & 8 ? c[1] : c[3];
      if constexpr (SIZE < 4) {
        const uint32_t v = off < 8 ? (off < 4 ? c[0] : c[1]) : (off < 12 ? c[2] : c[3]);   // the word that holds byte off
        if (h & 2) *reinterpret_cast<uint16_t*>(piece + (off & 12) + 2) = (uint16_t)(v >> 16);
        if (SIZE == 1 && (h & 1)) piece[off] = (uint8_t)(v >> (8 * (off & 3)));
      }
    }
    if (lane == 31 || next == 0) {   // bytes 0 to end % 16 - 1 of the last piece
      const int j = end >> 4, e = end & 15;
      uint32_t q[4] = {c[W], c[W + 1], c[W + 2], c[W + 3]};
      if (j < W / 4) {   // (the row's end)
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = j == k ? c[4 * k + i] : q[i];
        }
      }
      uint8_t* last = piece + 16 * j;
      if (e & 8) *reinterpret_cast<uint2*>(last) = make_uint2(q[0], q[1]);
      if (e & 4) *reinterpret_cast<uint32_t*>(last + (e & 8)) = e & 8 ? q[2] : q[0];
      if constexpr (SIZE < 4) {
        const uint32_t v = e & 8 ? (e & 4 ? q[3] : q[2]) : (e & 4 ? q[1] : q[0]);   // the word behind
        if (e & 2) *reinterpret_cast<uint16_t*>(last + (e & 12)) = (uint16_t)v;
        if (SIZE == 1 && (e & 1)) last[e - 1] = (uint8_t)(v >> (8 * (e & 2)));
      }
    }
  }
}

template <int AL, typename T>
__device__ __forceinline__ void store16(T* p, int n, const F2 (&v)[8]) {
  constexpr int WORDS = 4 * sizeof(T);
  uint32_t w[WORDS];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) {
      w[i] = pack2<T>(lo(v[i]), hi(v[i]));
    } else {
      w[2 * i] = __float_as_uint(lo(v[i]));
      w[2 * i + 1] = __float_as_uint(hi(v[i]));
    }
  }
  if constexpr (AL == 0) {
    store_unaligned<WORDS, sizeof(T)>(p, n, w);
  } else if constexpr (AL == 2) {
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < WORDS; i += 8) st32(reinterpret_cast<uint32_t*>(p) + i, *reinterpret_cast<uint32_t(*)[8]>(w + i));
    }
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4)
      if (i < WORDS / 2 ? n > 0 : n > 8) reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// 16 elements of the weight [K] from `at` on
template <int AL>
__device__ __forceinline__ void load_weight(const void* p, int type, int K, int at, F2 (&v)[8]) {
  if (type == ROW_BF16)
    load16<AL>(static_cast<const __nv_bfloat16*>(p) + at, K - at, p, 2ll * K, v);
  else if (type == ROW_FP16)
    load16<AL>(static_cast<const __half*>(p) + at, K - at, p, 2ll * K, v);
  else
    load16<AL>(static_cast<const float*>(p) + at, K - at, p, 4ll * K, v);
}

// ---------------------------------------------------------------------------
// quantization to e4m3
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The scale of a block, s = f32(amax / 448), and r = f32(1 / s) (1 for s = 0),
// from the bits of amax.  Straight-line: both quotients by Markstein's
// correction steps (see e4m3_quotient).  s: amax * f32(1/448) is within one
// unit in the last place of the quotient, 448 = 7 * 2^6 leaves the residual
// exact.  r: from the hardware's reciprocal, whose documented error is one unit
// in the last place, by one step; the step gives the correctly rounded value
// from any estimate within one unit, unless s has the largest significand.  (An
// error of 2^-23 relative would not do: where the significand of s is below 4/3
// that is up to 1.5 units, from which the step can miss.)  All 2^23
// significands of amax are tested.  `fast` says that s and r are what they
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

// The 8 codes of 4 pairs under the scale s: e4m3(f32(v / s)), 0 where s is 0;
// for blocks whose scale is `fast` ...
// The quotient, correctly rounded where the code depends on it, without the
// range test of e4m3_quotient: for r normal and |v / s| not above 2^9 the
// correction leaves every quotient below 2^-12 there (where each code is 0) and
// cannot overflow.  It is taken of -v, whose steps need no negation:
//   q = -v r,  e = q s + v  (= q s - (-v)),  q - e r;
// the codes' signs are flipped at the end, and a zero keeps its own.
__device__ __forceinline__ uint2 codes8_fast(const F2* v, float s, float r) {
  const F2 s2 = f2(s, s), nr = f2(-r, -r);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 q = mul2(v[i], nr);
    const F2 t = fma2(fma2(q, s2, v[i]), nr, q);
    c[i] = e4m3x2(lo(t), hi(t));
  }
  return s == 0.f ? make_uint2(0u, 0u) : make_uint2((c[0] | (c[1] << 16)) ^ 0x80808080u, (c[2] | (c[3] << 16)) ^ 0x80808080u);
}
// ... and for any scale, by the division (a NaN makes every code of its block
// NaN; in a block with an infinity the finite elements' codes are 0)
__device__ __forceinline__ uint2 codes8_any(const F2* v, float s) {
  uint32_t w[2] = {0u, 0u};
  if (s != 0.f) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const F2 a = h ? v[2] : v[0], b = h ? v[3] : v[1];
      const uint32_t x = e4m3x2(__fdiv_rn(lo(a), s), __fdiv_rn(hi(a), s)) | (e4m3x2(__fdiv_rn(lo(b), s), __fdiv_rn(hi(b), s)) << 16);
      if (h) w[1] = x;
      else w[0] = x;
    }
  }
  return make_uint2(w[0], w[1]);
}

// the larger magnitude, NaN if either is
__device__ __forceinline__ float amax2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Scale and codes of a warp's four blocks, 8 lanes each (the whole warp calls
// this).  A NaN makes the maximum and so the scale NaN.
__device__ __forceinline__ uint4 quantize_block(const F2 (&v)[8], float* s) {
  float a = amax2(lo(v[0]), hi(v[0])), b2 = amax2(lo(v[1]), hi(v[1]));
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    a = amax2(a, amax2(lo(v[i]), hi(v[i])));
    b2 = amax2(b2, amax2(lo(v[i + 1]), hi(v[i + 1])));
  }
  a = amax2(a, b2);
#pragma unroll
  for (int o = 4; o; o >>= 1) a = amax2(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  const BlockScale b = block_scale_of(__float_as_uint(a));
  uint2 c, d;
  if (__all_sync(0xFFFFFFFFu, b.fast)) {
    *s = b.s;
    c = codes8_fast(v, b.s, b.r);
    d = codes8_fast(v + 4, b.s, b.r);
  } else {
    *s = __fdiv_rn(a, 448.f);
    c = codes8_any(v, *s);
    d = codes8_any(v + 4, *s);
  }
  return make_uint4(c.x, c.y, d.x, d.y);
}

template <int AL>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint4 c) {
  if constexpr (AL == 2) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = c;
  } else if constexpr (AL == 1) {
    if (n > 0) *reinterpret_cast<uint2*>(p) = make_uint2(c.x, c.y);
    if (n > 8) *reinterpret_cast<uint2*>(p + 8) = make_uint2(c.z, c.w);
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    store_unaligned<4, 1>(p, n, w);
  }
}

// Vector `vec` (16 elements) of row `row`, n of which exist, to the output.
// The whole warp calls this, its lanes holding consecutive vectors from a
// multiple of 32 on.
template <int OUT, int AL>
__device__ __forceinline__ void emit16(const RowArgs& a, int row, int vec, int n, const F2 (&v)[8]) {
  const long long at = (long long)row * a.K + vec * 16;
  if constexpr (OUT == OUT_BLOCK) {
    float s;
    const uint4 c = quantize_block(v, &s);
    if (n > 0 && (vec & 7) == 0) a.scales[(long long)row * ((a.K + QBLOCK - 1) / QBLOCK) + (vec >> 3)] = s;
    store_codes<AL>(static_cast<uint8_t*>(a.out) + at, n, c);
  } else if constexpr (OUT == OUT_STATIC) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      w[h] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[h] |= (uint32_t)act_code_r(i & 1 ? hi(v[2 * h + i / 2]) : lo(v[2 * h + i / 2]), a.s_out, a.r_out) << (8 * i);
    }
    store_codes<AL>(static_cast<uint8_t*>(a.out) + at, n, make_uint4(w[0], w[1], w[2], w[3]));
  } else if constexpr (OUT == OUT_BF16) {
    store16<AL>(static_cast<__nv_bfloat16*>(a.out) + at, n, v);
  } else if constexpr (OUT == OUT_FP16) {
    store16<AL>(static_cast<__half*>(a.out) + at, n, v);
  } else {
    store16<AL>(static_cast<float*>(a.out) + at, n, v);
  }
}

// ---------------------------------------------------------------------------
// RMS norm:  r = x + residual,  y = r * w / sqrt(mean(r^2) + eps).
// The sum r is kept in fp32 for the norm (only the residual that is stored is
// rounded), so the output carries one rounding.  blockDim.x threads hold a
// row (NV vectors each, read once) and blockDim.y rows share a CTA, which
// goes on to the next rows with their loads already under way and the weight
// kept in registers.  NV = 0 reads the row twice, for rows that do not fit.
// residual_out may be the residual or x itself: every element is read by the
// warp that writes it, before it is written (store_unaligned writes a lane's
// last elements from the next lane, after both have theirs; what else a piece
// of load() covers is not used).
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

// The root is the hardware's (2 units), then two products, where a division by
// the square root would round once less: of 67 M codes of 16384 x 4096 rows 1353
// differ from the exact ones, with square root and division 1346.  (The row's
// sum and root in 64 bits left as many: the fp32 quotient of the codes'
// definition decides them.)
//
// MT: most threads a CTA has.  The registers are bounded for three CTAs of 256
// threads an SM (16384 x 4096 in 16 bits: 72.6 us, with two 79.3, with four 83.7).
// Rows that start anywhere (AL = 0) are bound by the instructions that shift
// them into place and by what is in flight: there the next row is not loaded
// ahead, which leaves registers for 768 threads an SM (8192 x 4099 in bf16:
// 88 us, loaded ahead 119; in fp32 116 and 124).  Under these bounds 40 of the
// instances spill 32 to 132 bytes a thread: those of rows that start anywhere in
// fp32, or in 16 bits with 1024 threads, and two fp32 vectors a thread.
template <typename T, int NV, int OUT, int AL, int MT>
__global__ void __launch_bounds__(MT, AL == 0 ? (MT < 768 ? 768 / MT : 1) : MT == 256 && NV == 1 && sizeof(T) == 2 ? 3 : 1) rmsnorm_kernel(const RowArgs a) {
  constexpr bool AHEAD = AL > 0;
  __shared__ float part[2][32];   // in turn, so that one barrier a row will do
  pdl_launch_dependents();
  pdl_wait();   // x, the residual and the weight may be the previous grid's output
  const int K = a.K;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* res_out = static_cast<T*>(a.res_out);
  const int step = gridDim.x * blockDim.y;
  if constexpr (NV > 0) {
    const auto count = [&](long long row, int i) {
      return row < a.M ? K - ((int)threadIdx.x + i * (int)blockDim.x) * 16 : 0;
    };
    Raw16<AL, T> cx[NV], cr[NV];
    const auto fetch = [&](long long row) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = threadIdx.x + i * blockDim.x, n = count(row, i);
        cx[i].load(x + row * a.ldx + vec * 16, n, x, a.x_bytes);
        if (res) cr[i].load(res + row * K + vec * 16, n, res, a.row_bytes);
      }
    };
    long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if constexpr (AHEAD) fetch(row);
    F2 w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * blockDim.x;
      if (a.w) {
        load_weight<AL>(a.w, a.w_type, K, vec * 16, w[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = f2(1.f, 1.f);
      }
    }
    int turn = 0;
    // (the bound is of the CTA's first row: its threads meet in row_sum)
    for (long long first = (long long)blockIdx.x * blockDim.y; first < a.M; first += step, row += step, turn ^= 1) {
      F2 r[NV][8];
      if constexpr (!AHEAD) fetch(row);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        cx[i].values(r[i]);
        if (res) {
          F2 b[8];
          cr[i].values(b);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] = add2(r[i][j], b[j]);
        }
      }
      if (AHEAD && first + step < a.M) fetch(row + step);
      F2 sum = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = threadIdx.x + i * blockDim.x;
        if (res) store16<AL>(res_out + row * K + vec * 16, count(row, i), r[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma2(r[i][j], r[i][j], sum);
      }
      const float rs = rsqrtf(row_sum(lo(sum) + hi(sum), part[turn]) / (float)K + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = mul2(mul2(r[i][j], f2(rs, rs)), w[i][j]);
        emit16<OUT, AL>(a, (int)row, threadIdx.x + i * blockDim.x, count(row, i), r[i]);
      }
    }
  } else {
    int turn = 0;
    for (long long first = (long long)blockIdx.x * blockDim.y; first < a.M; first += step, turn ^= 1) {
      const long long row = first + threadIdx.y;
      const bool live = row < a.M;
      const auto load = [&](int vec, int n, F2 (&r)[8]) {
        load16<AL>(x + row * a.ldx + vec * 16, n, x, a.x_bytes, r);
        if (res) {
          F2 b[8];
          load16<AL>(res + row * K + vec * 16, n, res, a.row_bytes, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = add2(r[j], b[j]);
        }
      };
      const int rounds = (K + 16 * (int)blockDim.x - 1) / (16 * (int)blockDim.x);
      F2 r[8], sum = f2(0.f, 0.f);
      for (int i = 0; i < rounds; ++i) {
        const int vec = threadIdx.x + i * blockDim.x;
        load(vec, live ? K - vec * 16 : 0, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma2(r[j], r[j], sum);
      }
      const float rs = rsqrtf(row_sum(lo(sum) + hi(sum), part[turn]) / (float)K + a.eps);
      for (int i = 0; i < rounds; ++i) {
        const int vec = threadIdx.x + i * blockDim.x;
        const int n = live ? K - vec * 16 : 0;
        load(vec, n, r);
        if (res) store16<AL>(res_out + row * K + vec * 16, n, r);
        F2 w[8];
        if (a.w) {
          load_weight<AL>(a.w, a.w_type, K, vec * 16, w);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = f2(1.f, 1.f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = mul2(mul2(r[j], f2(rs, rs)), w[j]);
        emit16<OUT, AL>(a, (int)row, vec, n, r);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gated SiLU  y = g / (1 + e^-g) * u,  and (GATE = false) the plain copy that
// the activation quantizer is.  A warp takes 32 vectors of a row at a time
// (`parts` of them a row), the next ones' loads under way.
// ---------------------------------------------------------------------------
// FAST (outputs of 16 or 8 bits): the hardware's exponential and reciprocal.
// Their error, about 2^-22 plus 2^-24 per unit of |g|, stays far below half a
// step of the output.  For g down to GATE_TAIL: below -87.3 the reciprocal of
// 1 + e^-g would be flushed to 0, below -88.7 e^-g overflows, while a large u
// makes the result an ordinary number still.
constexpr float GATE_TAIL = -80.f;
template <bool FAST>
__device__ __forceinline__ F2 silu_mul2(F2 g, F2 u) {
  if constexpr (FAST) {
    const F2 t = mul2(g, f2(-1.44269504f, -1.44269504f));   // log2 e
    float e0, e1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(lo(t)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(hi(t)));
    const F2 d = add2(f2(e0, e1), f2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(lo(d)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(hi(d)));
    return mul2(mul2(g, f2(r0, r1)), u);
  } else {
    return f2(lo(g) / (1.f + expf(-lo(g))) * lo(u), hi(g) / (1.f + expf(-hi(g))) * hi(u));
  }
}
// For g < GATE_TAIL 1 + e^-g is e^-g in fp32, so the result is g e^g u: taken in
// four factors of e^(g/4), each of them (g > -349) and every partial product
// that a result within fp32 has an ordinary number.  FAST: within 2^-20 plus
// 2^-23 per unit of |g|.
template <bool FAST>
__device__ __forceinline__ float silu_mul_tail(float g, float u) {
  float h;
  if constexpr (FAST) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(g * (0.25f * 1.44269504f)));
  else h = expf(0.25f * g);
  return (g * h * h) * (u * h * h);
}
// Whether one of 16 packed elements may lie below GATE_TAIL, from their bits: as
// unsigned numbers those of negative values grow with the magnitude (a NaN
// with a sign counts too).  Three-way maxima of whole words: 6 instructions for
// 16 elements in 16 bits, where minima of the numbers are 15 (8192 x 14336 to
// static codes, bound by issue: 102 us, by minima 105; without this test 101).
template <typename T, int N>
__device__ __forceinline__ bool tail_among(const uint32_t (&t)[N]) {
  uint32_t m = t[0];
  if constexpr (sizeof(T) == 4) {
    m = max(m, t[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) m = __vimax3_u32(m, t[i], t[i + 1]);
    return m > 0xC2A00000u;
  } else {
    constexpr uint32_t limit = std::is_same<T, __half>::value ? 0xD500D500u : 0xC2A0C2A0u;   // -80 twice
    m = __vimax3_u16x2(m, t[1], limit);
#pragma unroll
    for (int i = 2; i < N; i += 2) m = __vimax3_u16x2(m, t[i], t[i + 1]);
    return m != limit;
  }
}
// v = silu(v) * w of 16 elements; TAIL: some of them may be below GATE_TAIL.
// What an element becomes does not depend on the others.
template <bool FAST, bool TAIL>
__device__ __forceinline__ void silu_mul16(F2 (&v)[8], const F2 (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const F2 y = silu_mul2<FAST>(v[i], w[i]);
    if constexpr (TAIL)
      v[i] = f2(lo(v[i]) < GATE_TAIL ? silu_mul_tail<FAST>(lo(v[i]), lo(w[i])) : lo(y),
                hi(v[i]) < GATE_TAIL ? silu_mul_tail<FAST>(hi(v[i]), hi(w[i])) : hi(y));
    else
      v[i] = y;
  }
}

// The gate's registers are bounded for three CTAs an SM, in static codes four
// (102 us where three take 105; to bf16 three take 107 us and four 115): without
// a bound the tail, which hardly any call reaches, sets their number.
template <typename T, bool GATE, int OUT, int AL>
__global__ void __launch_bounds__(256, !GATE || sizeof(T) == 4 || OUT == OUT_FP32 ? 1 : AL == 2 && OUT == OUT_STATIC ? 4 : 3) rows_kernel(const RowArgs a, int parts) {
  pdl_launch_dependents();
  pdl_wait();
  const T* x = static_cast<const T*>(a.x);
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (blockDim.x >> 5), warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int dr = warps / parts, dp = warps - dr * parts;   // one step, in rows and parts
  long long row = warp / parts;
  int part = warp - (int)row * parts;
  Raw16<AL, T> g, u;
  const auto fetch = [&] {
    if (row < a.M) {
      const int at = (part * 32 + lane) * 16, n = a.K - at;
      g.load(x + row * a.ldx + at, n, x, a.x_bytes);
      if constexpr (GATE) u.load(x + row * a.ldx + a.K + at, n, x, a.x_bytes);
    }
  };
  fetch();
  while (row < a.M) {
    F2 v[8], w[8];
    bool tail = false;
    if constexpr (GATE) {
      uint32_t t[Raw16<AL, T>::PACKED];
      g.words(t);
      tail = tail_among<T>(t);
      Raw16<AL, T>::unpack(t, v);
      u.values(w);
    } else {
      g.values(v);
    }
    const long long r = row;
    const int vec = part * 32 + lane;
    row += dr;
    part += dp;
    if (part >= parts) {
      part -= parts;
      ++row;
    }
    fetch();
    // (two ways out: where they meet before emit16 the compiler cannot mix the
    // gate's instructions with the quantizer's, to static codes 113 us.  The
    // test behind the loop, and what was written there done again: 96 us to
    // block codes; this way 92; without the test 91.)
    if constexpr (GATE) {
      if (__any_sync(0xFFFFFFFFu, tail)) {
        silu_mul16<OUT != OUT_FP32, true>(v, w);
        emit16<OUT, AL>(a, (int)r, vec, a.K - vec * 16, v);
        continue;
      }
      silu_mul16<OUT != OUT_FP32, false>(v, w);
    }
    emit16<OUT, AL>(a, (int)r, vec, a.K - vec * 16, v);
  }
}

}  // namespace dq
