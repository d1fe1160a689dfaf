// fp8q_fp4_math.cuh -- the arithmetic of 4-bit microscaled quantization shared
// by the quant kernels and the experts' GEMM epilogue: group scales, e2m1
// codes, and the place of a scale byte in its 128 x 4 block.
//
//   nvfp4 (groups of 16)  u = fl32(fl32(amax / 6) / g), sf = e4m3_rn(min(u, 448)),
//                         d = fl32(sf g), code = e2m1_rn(fl32(y / d)); d = 0: code 0
//   mxfp4 (groups of 32)  sf = fl32(max(amax, 1e-10) / 6) rounded up to a power of
//                         two, code = e2m1_rn(y / sf) (an exact product)
// Codes saturate at +-6, ties go to the even code, and every code keeps its
// value's sign.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp8q_common.cuh"
#include "fp8q_fp4.h"

namespace fp8q {

// The plan of up to kSmallPlan (token, slot) entries and the quantization of
// their tokens into the experts' rows, in one launch (arguments checked by the
// caller; E <= 512).
constexpr int kSmallPlan = 128;
fp8q_status moe_plan_quant_small(const void* x, int64_t T, int64_t H, int64_t ldx, const int* ids, int topk, int E,
                                 int format, const float* gscale, int* offsets, int* sf_offsets, int* pos, int* sf_row,
                                 void* q, uint8_t* sf, cudaStream_t stream);

namespace {   // internal linkage in every translation unit that includes it

constexpr int kNv = FP8Q_FP4_NV, kMx = FP8Q_FP4_MX;

template <int FMT>
__host__ __device__ constexpr int fp4_group() { return FMT == kNv ? 16 : 32; }

// Scale blocks of a row: 4 groups each.
__host__ __device__ inline int64_t fp4_kblocks(int fmt, int64_t K) {
  const int64_t span = fmt == kNv ? 64 : 128;
  return (K + span - 1) / span;
}

// Byte offset of the scale of (row, group) in a buffer of 512-byte blocks,
// kb blocks to a block row: row r of a block in lane r % 32, word r / 32 of
// that lane's 16 bytes, byte group % 4 -- what one tcgen05.cp of a block puts
// into tensor memory where the block-scaled MMA reads it.
__host__ __device__ inline int64_t fp4_sf_offset(int64_t row, int64_t group, int64_t kb) {
  return ((row >> 7) * kb + (group >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (group & 3);
}

// A group's scale byte and what its codes need: d = sf g and RN(1/d) (0 where
// d is 0, which makes every code 0).
struct Fp4Scale {
  uint32_t byte;
  float d, rcp;
};

// A tensor scale and its correctly rounded reciprocal.
struct Fp4G {
  float g, rcp;
};
__device__ __forceinline__ Fp4G fp4_g(const float* g) {
  const float v = g ? *g : 1.0f;
  return {v, __frcp_rn(v)};
}

// nvfp4: both quotients by Markstein's correction step, as in fp4_codes8 (1/6
// is rounded to nearest, too).  Its argument fails where a product under- or
// overflows: a tiny quotient becomes scale 0 either way, and of an infinite
// amax or quotient the minima make the largest scale (a NaN is dropped).
template <int FMT>
__device__ __forceinline__ Fp4Scale fp4_scale(float amax, const Fp4G& g) {
  Fp4Scale s;
  if constexpr (FMT == kNv) {
    constexpr float kSixth = 1.0f / 6.0f;
    const float a = fminf(amax, 3.40282347e38f);
    float u = a * kSixth;
    u = fmaf(fmaf(-6.0f, u, a), kSixth, u);
    float q = u * g.rcp;
    q = fminf(fmaf(fmaf(-g.g, q, u), g.rcp, q), 448.0f);
    s.byte = static_cast<uint32_t>(__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3));
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(s.byte), __NV_E4M3);
    s.d = __fmul_rn(__half2float(__half(h)), g.g);
    s.rcp = s.d > 0.0f ? __frcp_rn(s.d) : 0.0f;
  } else {
    // fl32(max(amax, 1e-10) / 6) >= 2^-36 is a positive normal; its exponent,
    // one up unless it is a power of two.  2^127 (byte 254) is the largest.
    const uint32_t u = __float_as_uint(__fdiv_rn(fmaxf(amax, 1e-10f), 6.0f));
    uint32_t b = (u + 0x007FFFFFu) >> 23;
    if (b > 254u) b = 254u;
    s.byte = b;
    s.d = __uint_as_float(b << 23);
    // 2^-(b - 127): b = 254 would be 2^-127, a subnormal
    s.rcp = b < 254u ? __uint_as_float((254u - b) << 23) : __uint_as_float(0x00400000u);
  }
  return s;
}

// Eight values -> eight codes, value 0 in the lowest four bits.  nvfp4: the
// IEEE quotient fl32(y / d) by Markstein's division step (q0 = RN(y rcp), the
// residual y - q0 d exact under FMA, RN(q0 + r rcp) = RN(y / d) for
// rcp = RN(1/d)); a quotient too small for that argument rounds to code 0
// either way.  The residual is taken as q0 d - y and subtracted, so that a zero
// quotient, of y = -0 or d = 0 too, keeps the sign of y.  mxfp4: rcp is a power
// of two, the product is the quotient.
// `far`: some quotient may be infinite (or of an infinite y), where that
// residual would be NaN: the minimum, which drops a NaN, gives the saturated
// code, and the sign is copied.
// (Pairs of fp32 operations, .f32x2, were no faster: they cost the moves that
// pair the registers.)
template <int FMT>
__device__ __forceinline__ bool fp4_far(float amax, const Fp4Scale& s) {
  return FMT == kNv && !(amax * s.rcp < 0x1p100f);
}
__device__ __forceinline__ uint32_t fp4_cvt8(const float (&q)[8]) {
  uint32_t c;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(c)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return c;
}
template <int FMT>
__device__ __forceinline__ uint32_t fp4_codes8(const float* y, const Fp4Scale& s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = y[i] * s.rcp;
    if constexpr (FMT == kNv) q[i] = fmaf(-fmaf(q[i], s.d, -y[i]), s.rcp, q[i]);
  }
  return fp4_cvt8(q);
}
__device__ __forceinline__ uint32_t fp4_codes8_far(const float* y, const Fp4Scale& s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = y[i] * s.rcp;
    q[i] = copysignf(fminf(fabsf(fmaf(fmaf(-v, s.d, y[i]), s.rcp, v)), 8.0f), y[i]);
  }
  return fp4_cvt8(q);
}

// One value's code, in the low four bits.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_code1(float y, const Fp4Scale& s) {
  float v = y * s.rcp;
  if constexpr (FMT == kNv) v = fminf(fabsf(fmaf(fmaf(-v, s.d, y), s.rcp, v)), 8.0f);
  uint32_t c;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "mov.b32 %0, {b, 0, 0, 0};\n\t}"
      : "=r"(c)
      : "f"(copysignf(v, y)), "f"(0.0f));
  return c;
}

// fp32 silu(g) u: e = 2^(-g log2 e) by ex2.approx of the rounded product plus
// its exact residual (first order), one rounding of 1 + e, a division good to
// 2 ulp and a product: relative error below 2^-20 for |g| <= 85.  Beyond, e over- or
// underflows: g / inf = -0 and g / 1 are the limits (below -85 silu itself is less
// than 2^-116, below -87.3, where __fdividef gives 0, less than 2^-119).  The
// residual term is dropped there (0 inf would be NaN).
__device__ __forceinline__ float silu_mul_f32(float g, float u) {
  const float L2E = 1.44269502f;           // fl32(log2 e)
  const float L2E_LO = 1.925963e-8f;       // log2 e - L2E
  const float a = -g * L2E;
  float lo = fmaf(-g, L2E, -a);
  lo = fmaf(-g, L2E_LO, lo);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
  if (fabsf(g) <= 85.0f) e = fmaf(e, lo * 0.693147182f, e);
  return __fdividef(g, 1.0f + e) * u;
}

}  // namespace
}  // namespace fp8q
