// fp8q_fp4_quant.cu -- 4-bit microscaled quantization (nvfp4, mxfp4) of bf16
// rows, plain or fused with its producer (RMSNorm, SiLU*mul), its scatter into
// the experts' rows, and the way back to values.
//
// HBM-bound: a row's values are read once (2 bytes each, SiLU*mul 4) and
// leave as half a byte each plus a scale byte per group.  The unit of work is
// an item of 16 neighbouring values of a row, one 32-byte load: an nvfp4
// group, or half an mxfp4 one (the two halves sit in neighbouring lanes and
// exchange their amax by one shuffle).  y is the exact bf16 value of its
// definition, as in the FP8 quant kernels (the same brackets, the same rare
// fp64 recomputation), so codes and scales equal the definition bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8q_common.cuh"
#include "fp8q_fp4_math.cuh"
#include "fp8q_quant_math.cuh"

namespace fp8q {
namespace {

enum { OP_PLAIN = 0, OP_SILU = 1 };

struct Fp4QuantParams {
  const uint16_t* x;         // bf16 [M, K] ([M, 2K] = [gate | up] for SiLU), leading dimension ldx
  int64_t M, K, ldx;
  const uint16_t* w;         // RMSNorm weight [K]
  float eps;
  const float* g;            // tensor scale or null
  uint8_t* q;                // codes, ldq bytes a row
  int64_t ldq;
  uint8_t* sf;               // scale blocks, kb to a block row
  int64_t kb;
  const int* pos;            // scatter: [M, topk] destination rows (negative: none) and scale rows
  const int* sf_row;
  int topk;
};

// Items are 16 values: two 16-byte chunks of 8.
struct Item {
  uint4 a, b;
};

__device__ __forceinline__ Item ld_item(const uint16_t* p, bool wide) {
  Item v;
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y), "=r"(v.b.z),
                   "=r"(v.b.w)
                 : "l"(p));
  } else {
    v.a = __ldg(reinterpret_cast<const uint4*>(p));
    v.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  return v;
}

__device__ __forceinline__ void st_item(uint16_t* p, const uint32_t (&o)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                 "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Both ends of the bracket of bf16(silu(g) u) (the bounds of silu_pair) in the
// lanes of a word: lo and hi, bf16, |lo| <= |y| <= |hi|.
__device__ __forceinline__ void silu_bracket(uint32_t gw, uint32_t uw, uint32_t& lo, uint32_t& hi) {
  const uint64_t g2 = bf2_to_f2(gw);
  const uint64_t np = mul2(mul2(g2, neg_sigmoid2(g2)), bf2_to_f2(uw));          // -silu(g) u
  lo = f2_to_bf2_rn(mul2(np, dup2(-kSiluLo)));
  hi = f2_to_bf2_rn(mul2(np, dup2(-kSiluHi)));
}

// The exact values of a chunk.
__device__ __noinline__ uint4 silu_chunk_exact(const uint4 g, const uint4 u) {
  uint4 lo, hi;
  silu_bracket(g.x, u.x, lo.x, hi.x);
  silu_bracket(g.y, u.y, lo.y, hi.y);
  silu_bracket(g.z, u.z, lo.z, hi.z);
  silu_bracket(g.w, u.w, lo.w, hi.w);
  return silu_chunk_fix(g, u, lo);
}

// The bracket of a chunk; tested on the packed bf16 words, whose magnitudes are
// ordered as integers:
// - gates below -60, where |silu| <= 60 e^-60 < 2^-80: a signed zero, whose
//   code is the value's unless the whole group is nearly as small; `wide`
//   gathers the bound 2^-80 |up|.  (Exact values for them, as heavy-tailed
//   gates have them one in 4000, took a seventh of the kernel's time.)
// - other values or gates so small that the bracket does not serve, and gates
//   above 2^127, whose exponential's argument may overflow: exact at once.
__device__ __forceinline__ uint4 silu_chunk(const uint4& g, const uint4& u, uint4& hi, float& wide) {
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
  constexpr uint32_t kMag = 0x7FFF7FFFu, k60 = 0x4270u, kNeg60 = 0xC270u, kSmall = (127 - 99) << 7;   // bf16 bits
  constexpr int kHuge = 0x7F00;            // 2^127
  uint32_t lo[4], h[4], gm[4], least = kMag;      // smallest magnitude of gates and lower ends
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    silu_bracket(gw[k], uw[k], lo[k], h[k]);
    gm[k] = gw[k] & kMag;
    least = __vimin3_u16x2(least, gm[k], lo[k] & kMag);
  }
  const uint32_t most = __vmaxu2(__vimax3_u16x2(gm[0], gm[1], gm[2]), gm[3]);       // the gate furthest from 0
  // a lower end of 2^-99 at least comes from a p above 2^-100
  bool small = min(least & 0xFFFFu, least >> 16) < kSmall;
  if (small || max(most & 0xFFFFu, most >> 16) > k60) {
    const uint32_t low = __vmaxu2(__vimax3_u16x2(gw[0], gw[1], gw[2]), gw[3]);      // the lowest negative gate
    if (max(low & 0xFFFFu, low >> 16) > kNeg60) {
      uint32_t largest = 0;                // up of such a gate
      least = kMag;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t far = __vcmpgtu2(gw[k], kNeg60 * 0x10001u), zero = ~uw[k] & 0x80008000u & far;
        lo[k] = (lo[k] & ~far) | zero;
        h[k] = (h[k] & ~far) | zero;
        largest = __vmaxu2(largest, uw[k] & kMag & far);
        least = __vimin3_u16x2(least, gm[k] | far, (lo[k] & kMag) | far);
      }
      wide = fmaxf(wide, bf16_bits_to_f32(max(largest & 0xFFFFu, largest >> 16)) * 0x1p-80f);
      small = min(least & 0xFFFFu, least >> 16) < kSmall;
    }
    const uint32_t top = __vmaxs2(__vimax3_s16x2(gw[0], gw[1], gw[2]), gw[3]);      // the largest gate
    small |= max(static_cast<int16_t>(top & 0xFFFFu), static_cast<int16_t>(top >> 16)) > kHuge;
  }
  uint4 y = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  if (small) hi = y = silu_chunk_exact(g, u);
  return y;
}

__device__ __forceinline__ bool differ(const uint4& a, const uint4& b) {
  return ((a.x ^ b.x) | (a.y ^ b.y) | (a.z ^ b.z) | (a.w ^ b.w)) != 0;
}

__device__ __forceinline__ void chunk_to_f32(const uint4& c, float* f) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Codes and scale of one item, y already bf16.  mxfp4: every lane of a pair
// must call it (shuffle); a lane without an item passes zeros.
template <int FMT>
__device__ __forceinline__ uint2 item_codes(const Item& y, const Fp4G& g, Fp4Scale& s, float& amax) {
  amax = absmax2_to_f32(chunk_absmax2(y.b, chunk_absmax2(y.a, 0u)));
  if constexpr (FMT == kMx) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  s = fp4_scale<FMT>(amax, g);
  float f[8];
  uint2 c;
  chunk_to_f32(y.a, f);
  c.x = fp4_codes8<FMT>(f, s);
  chunk_to_f32(y.b, f);
  c.y = fp4_codes8<FMT>(f, s);
  if (fp4_far<FMT>(amax, s)) {
    c.y = fp4_codes8_far(f, s);
    chunk_to_f32(y.a, f);
    c.x = fp4_codes8_far(f, s);
  }
  return c;
}
template <int FMT>
__device__ __forceinline__ uint2 item_codes(const Item& y, const Fp4G& g, uint32_t* byte) {
  Fp4Scale s;
  float amax;
  const uint2 c = item_codes<FMT>(y, g, s, amax);
  *byte = s.byte;
  return c;
}

// Store item `it` (of K / 16) of a row: its codes at row `row`, its group's
// scale at scale row `srow`; the last item of a row also zeroes the bytes of
// the groups that fill its last scale block.
template <int FMT>
__device__ __forceinline__ void store_item(const Fp4QuantParams& p, int64_t row, int64_t srow, int it, int items,
                                           const uint2& c, uint32_t byte) {
  *reinterpret_cast<uint2*>(p.q + row * p.ldq + 8 * it) = c;
  const int group = FMT == kNv ? it : it >> 1;
  if (FMT == kNv || (it & 1) == 0) p.sf[fp4_sf_offset(srow, group, p.kb)] = static_cast<uint8_t>(byte);
  if (it == items - 1)
    for (int j = group + 1; j & 3; ++j) p.sf[fp4_sf_offset(srow, j, p.kb)] = 0;
}

template <int FMT>
__device__ __forceinline__ void emit_item(const Fp4QuantParams& p, int64_t row, int it, int items, const uint2& c,
                                          uint32_t byte) {
  if (p.pos == nullptr) {
    store_item<FMT>(p, row, row, it, items, c, byte);
  } else {
    for (int j = 0; j < p.topk; ++j) {
      const int dst = __ldg(p.pos + row * p.topk + j);
      if (dst >= 0) store_item<FMT>(p, dst, __ldg(p.sf_row + row * p.topk + j), it, items, c, byte);
    }
  }
}

// Row of item i of `total`; a 32-bit division where it serves.
__device__ __forceinline__ int64_t item_row(int64_t i, int items, int64_t total) {
  return total <= 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(items))
                             : i / items;
}

// Plain and SiLU*mul: independent items, one a thread and step.  A warp takes 32
// neighbouring items: their scale bytes lie in 8 blocks, a sector each.  (Eight
// rows by four items instead, whose scales fill one sector, were slower: 70
// against 65 us for 8192 x 12288 plain values.)
constexpr int kItemThreads = 256;

template <int FMT, int OP>
__global__ void __launch_bounds__(kItemThreads, OP == OP_SILU ? 4 : 6)
    fp4_items_kernel(const Fp4QuantParams p, int wide) {
  const int items = static_cast<int>(p.K >> 4);
  const int64_t total = p.M * items;
  griddep_wait();
  griddep_launch_dependents();
  const Fp4G g = fp4_g(p.g);
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kItemThreads;
  // whole warps stay in the loop: total is even, so pairs of lanes live and end together
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kItemThreads + (threadIdx.x & ~31); i0 < total; i0 += stride) {
    const int64_t i = i0 + lane;
    const bool live = i < total;
    const int64_t row = live ? item_row(i, items, total) : 0;
    const int it = live ? static_cast<int>(i - row * items) : 0;
    const Item zero = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    Item y = zero;
    uint32_t byte;
    uint2 c;
    if constexpr (OP == OP_SILU) {
      // Where the two ends of a value's bracket give the same codes and scale,
      // so does the value between them (both are monotone): the exact value,
      // an fp64 chain of some thousand cycles, is needed only where they do not
      // (one in ~50 of the open brackets, themselves 5e-4 of the values).  What
      // bounds the kernel is its instructions, 34 a value (8192 x 12288 nvfp4:
      // 128 us of normal values, 135 of heavy-tailed ones, 53% of HBM).  Tried
      // and slower: a wider and cheaper bracket, whose ends are both coded for
      // every value (by 10%); open values coded pair by pair, each behind a vote
      // (6%); three or five CTAs an SM (167, 152 with spills, when four took 153).
      Item hi = zero;
      float bound = 0.0f;               // bound of the values that y has as zeros
      const uint16_t* x = p.x + row * p.ldx + 16 * it;
      if (live) {
        const Item gate = ld_item(x, wide), up = ld_item(x + p.K, wide);
        y.a = silu_chunk(gate.a, up.a, hi.a, bound);
        y.b = silu_chunk(gate.b, up.b, hi.b, bound);
      }
      Fp4Scale s;
      float amax;
      c = item_codes<FMT>(y, g, s, amax);
      byte = s.byte;
      const bool open = differ(y.a, hi.a) || differ(y.b, hi.b);
      // a value below d / 5 has code 0; one of at most amax leaves the scale
      const bool low = bound > 0.0f && (bound > amax || (s.d > 0.0f && bound >= 0.2f * s.d));
      if (__any_sync(0xFFFFFFFFu, open || low)) {
        uint32_t byte2;
        const uint2 c2 = item_codes<FMT>(hi, g, &byte2);
        if (__any_sync(0xFFFFFFFFu, low || byte != byte2 || c.x != c2.x || c.y != c2.y)) {
          if (open || low) {            // its inputs again, rather than in registers all along
            const Item gate = ld_item(x, wide), up = ld_item(x + p.K, wide);
            y.a = silu_chunk_exact(gate.a, up.a);
            y.b = silu_chunk_exact(gate.b, up.b);
          }
          c = item_codes<FMT>(y, g, &byte);
        }
      }
    } else {
      if (live) y = ld_item(p.x + row * p.ldx + 16 * it, wide);
      c = item_codes<FMT>(y, g, &byte);
    }
    if (live) emit_item<FMT>(p, row, it, items, c, byte);
  }
}

// RMSNorm: one CTA a row.  y = bf16(bf16(x r) w), r = 1/sqrt(mean(x^2) + eps);
// the sum of squares in fp64.  IT items a thread stay in registers between the
// two passes; IT = 0 (rows of any length) reads them again.
template <int FMT, int IT>
__global__ void __launch_bounds__(512, IT == 4 ? 1 : 2) fp4_rms_kernel(const Fp4QuantParams p, int wide) {
  __shared__ double red[32];
  const int items = static_cast<int>(p.K >> 4);
  const int T = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Item zero = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  griddep_wait();
  griddep_launch_dependents();
  const Fp4G g = fp4_g(p.g);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const uint16_t* x = p.x + row * p.ldx;
    Item v[IT ? IT : 1];
    double ss = 0.0;
    auto add = [&](const Item& a) {
      float f[16];
      chunk_to_f32(a.a, f);
      chunk_to_f32(a.b, f + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = __fma_rn(static_cast<double>(f[i]), static_cast<double>(f[i]), ss);
    };
    if constexpr (IT > 0) {
#pragma unroll
      for (int k = 0; k < IT; ++k) v[k] = tid + k * T < items ? ld_item(x + 16 * (tid + k * T), wide) : zero;
#pragma unroll
      for (int k = 0; k < IT; ++k) add(v[k]);
    } else {
      for (int it = tid; it < items; it += T) add(ld_item(x + 16 * it, wide));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    __syncthreads();                       // red is free again
    if (lane == 0) red[warp] = ss;
    __syncthreads();
    ss = 0.0;
    for (int i = 0; i < (T >> 5); ++i) ss += red[i];
    float r_lo, r_hi;
    rms_bracket(ss / static_cast<double>(p.K) + static_cast<double>(p.eps), r_lo, r_hi);
    const uint64_t rlo2 = dup2(r_lo), rhi2 = dup2(r_hi);
    auto norm = [&](const uint4& xv, const uint4& wv) {
      uint32_t d = 0;
      uint4 y;
      y.x = bf2_mul(rms_n_pair(xv.x, rlo2, rhi2, d), wv.x);
      y.y = bf2_mul(rms_n_pair(xv.y, rlo2, rhi2, d), wv.y);
      y.z = bf2_mul(rms_n_pair(xv.z, rlo2, rhi2, d), wv.z);
      y.w = bf2_mul(rms_n_pair(xv.w, rlo2, rhi2, d), wv.w);
      return d ? rms_chunk_fix(xv, wv, y, rlo2, rhi2, ss, p.K, p.eps) : y;
    };
    const int steps = IT ? IT : (items + T - 1) / T;
#pragma unroll
    for (int k = 0; k < steps; ++k) {
      const int it = tid + k * T;
      const bool live = it < items;
      Item y = zero;
      if (live) {
        const Item a = IT ? v[IT ? k : 0] : ld_item(x + 16 * it, wide);
        const uint4* wp = reinterpret_cast<const uint4*>(p.w) + 2 * it;
        y.a = norm(a.a, __ldg(wp));
        y.b = norm(a.b, __ldg(wp + 1));
      }
      uint32_t byte;
      const uint2 c = item_codes<FMT>(y, g, &byte);
      if (live) store_item<FMT>(p, row, row, it, items, c, byte);
    }
  }
}

// Values: bf16_rn(fl32(fl32(code sf) g)), an item a thread and step, stored at
// once where rows allow it: 8192 x 12288 in 42 us (6.1 TB/s); as two 16-byte
// halves, each of half a sector, 60.  (Two or four items a step: 4096 x 4096
// from 8.8 to 10.6 and 14.4 us.)
template <int FMT>
__global__ void __launch_bounds__(kItemThreads)
    fp4_dequant_kernel(const uint8_t* q, int64_t ldq, const uint8_t* sf, int64_t kb, const float* gp, int64_t M,
                       int64_t K, uint16_t* y, int64_t ldy, int wide) {
  const int items = static_cast<int>(K >> 4);
  const int64_t total = M * items;
  griddep_wait();
  griddep_launch_dependents();
  const float g = gp ? *gp : 1.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kItemThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kItemThreads) {
    const int64_t row = item_row(i, items, total);
    const int it = static_cast<int>(i - row * items);
    const uint2 c = *reinterpret_cast<const uint2*>(q + row * ldq + 8 * it);
    const uint32_t b = sf[fp4_sf_offset(row, FMT == kNv ? it : it >> 1, kb)];
    float s;
    if constexpr (FMT == kNv) {
      s = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
    } else {
      s = b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);   // 255 -> infinity
      if (b == 255u) s = __uint_as_float(0x7FFFFFFFu);                   // E8M0 NaN
    }
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t h2;
      const uint16_t byte = static_cast<uint16_t>(((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu);
      asm("{\n\t.reg .b8 lo, hi;\n\t"
          "mov.b16 {lo, hi}, %1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, lo;\n\t}"
          : "=r"(h2)
          : "h"(byte));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      const __nv_bfloat162 v = __floats2bfloat162_rn(__fmul_rn(__fmul_rn(f.x, s), g), __fmul_rn(__fmul_rn(f.y, s), g));
      o[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    st_item(y + row * ldy + 16 * it, o, wide);
  }
}

// ------------------------------------------------- few tokens of experts' rows
// Plan and quantization together, a CTA a token: with at most kSmallPlan
// entries every CTA counts them all itself.  An expert then has at most one
// block row of scales, so an entry's scales lie in the block row that counts
// the experts present before its own.  Two launches took 5.6 us for a token.
template <int FMT>
__global__ void __launch_bounds__(kItemThreads)
    moe_small_kernel(Fp4QuantParams p, const int* ids, int E, int* offsets, int* sf_offsets, int* pos, int* sf_row,
                     int wide) {
  __shared__ int id[kSmallPlan], row_of[kSmallPlan], srow_of[kSmallPlan];
  __shared__ uint32_t present[16];                      // a bit for each expert with entries
  const int n = static_cast<int>(p.M) * p.topk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 16) present[tid] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const Fp4G g = fp4_g(p.g);
  if (tid < n) {
    int e = __ldg(ids + tid);
    if (e < 0 || e >= E) e = -1;
    id[tid] = e;
    if (e >= 0) atomicOr(&present[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  // entries of experts before e, and of e before entry `upto`
  auto below = [&](int e, int upto) {
    int c = 0;
    for (int i = 0; i < n; ++i) c += (id[i] >= 0 && id[i] < e) || (id[i] == e && i < upto);
    return c;
  };
  auto blocks_below = [&](int e) {
    int c = 0;
    for (int w = 0; w <= (e - 1) >> 5; ++w)
      c += __popc(w == e >> 5 ? present[w] & ((1u << (e & 31)) - 1u) : present[w]);
    return c;
  };
  const int64_t t = blockIdx.x;
  if (warp == 0) {
    for (int j = lane; j < p.topk; j += 32) {
      const int i = static_cast<int>(t) * p.topk + j, e = id[i];
      row_of[j] = e >= 0 ? below(e, i) : -1;
      // the rank within the expert: rows before it less those of experts before
      srow_of[j] = e >= 0 ? 128 * blocks_below(e) + row_of[j] - below(e, 0) : -1;
      pos[i] = row_of[j];
      sf_row[i] = srow_of[j];
    }
  } else if (t == 0) {
    for (int e = tid - 32; e <= E; e += kItemThreads - 32) {
      offsets[e] = below(e, 0);
      sf_offsets[e] = blocks_below(e);
    }
  }
  __syncthreads();
  const int items = static_cast<int>(p.K >> 4);
  const Item zero = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  for (int i0 = tid & ~31; i0 < items; i0 += kItemThreads) {
    const int it = i0 + lane;
    const bool live = it < items;
    const Item y = live ? ld_item(p.x + t * p.ldx + 16 * it, wide) : zero;
    uint32_t byte;
    const uint2 c = item_codes<FMT>(y, g, &byte);
    if (live)
      for (int j = 0; j < p.topk; ++j)
        if (row_of[j] >= 0) store_item<FMT>(p, row_of[j], srow_of[j], it, items, c, byte);
  }
}

// ------------------------------------------------------------------ host side

// Blocks of the item kernels: enough that each thread has about one item, but
// no more than 16 resident blocks' worth a pass (they stride).
unsigned item_blocks(int64_t total) {
  int64_t b = (total + kItemThreads - 1) / kItemThreads;
  const int64_t cap = static_cast<int64_t>(num_sms()) * 32;
  return static_cast<unsigned>(b < cap ? b : cap);
}

template <int FMT, int OP>
fp8q_status launch_items(const Fp4QuantParams& p, cudaStream_t stream) {
  const int wide = aligned(p.x, 32) && p.ldx % 16 == 0;
  return launch_kernel(fp4_items_kernel<FMT, OP>, dim3(item_blocks(p.M * (p.K >> 4))), dim3(kItemThreads), 0, stream,
                       1, p, wide);
}

template <int FMT>
fp8q_status launch_rms(const Fp4QuantParams& p, cudaStream_t stream) {
  const int wide = aligned(p.x, 32) && p.ldx % 16 == 0;
  const int64_t items = p.K >> 4;
  // Few rows: an item a thread, for the shortest row.  Many: two, and four
  // where that takes over 512 threads, in short CTAs, so that many rows are in
  // flight on an SM and cover each other's reductions.
  const int it = items <= 512 && p.M <= 4 * num_sms() ? 1 : items <= 1024 ? 2 : items <= 2048 ? 4 : 0;
  const int64_t need = it ? (items + it - 1) / it : 512;
  const int T = static_cast<int>((need + 31) / 32 * 32);
  const int64_t cap = static_cast<int64_t>(num_sms()) * (2048 / T) * 4;
  const dim3 grid(static_cast<unsigned>(p.M < cap ? p.M : cap)), block(T);
  switch (it) {
    case 1: return launch_kernel(fp4_rms_kernel<FMT, 1>, grid, block, 0, stream, 1, p, wide);
    case 2: return launch_kernel(fp4_rms_kernel<FMT, 2>, grid, block, 0, stream, 1, p, wide);
    case 4: return launch_kernel(fp4_rms_kernel<FMT, 4>, grid, block, 0, stream, 1, p, wide);
    default: return launch_kernel(fp4_rms_kernel<FMT, 0>, grid, block, 0, stream, 1, p, wide);
  }
}

// Sizes and pointers shared by the quant entry points; *go is set when there
// is work to launch.
fp8q_status check_quant(const void* x, int64_t M, int64_t K, int64_t width, int64_t ldx, int format, const float* g,
                        const void* q, int64_t ldq, const void* sf, bool* go) {
  *go = false;
  if (format != FP8Q_FP4_NV && format != FP8Q_FP4_MX) return FP8Q_ERR_INVALID_ARG;
  if (M < 0 || K <= 0 || K % 32 != 0 || K > (int64_t{1} << 30) || M >= (int64_t{1} << 31)) return FP8Q_ERR_INVALID_ARG;
  if (ldx < width || ldx % 8 != 0 || ldq < K / 2 || ldq % 8 != 0) return FP8Q_ERR_INVALID_ARG;
  if (format == FP8Q_FP4_MX && g) return FP8Q_ERR_INVALID_ARG;
  if (M == 0) return FP8Q_OK;
  if (!x || !q || !sf) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16) || !aligned(g, 4)) return FP8Q_ERR_INVALID_ARG;
  *go = true;
  return FP8Q_OK;
}

Fp4QuantParams quant_params(const void* x, int64_t M, int64_t K, int64_t ldx, int format, const float* g, void* q,
                            int64_t ldq, uint8_t* sf) {
  Fp4QuantParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.M = M;
  p.K = K;
  p.ldx = ldx;
  p.g = g;
  p.q = static_cast<uint8_t*>(q);
  p.ldq = ldq;
  p.sf = sf;
  p.kb = fp4_kblocks(format, K);
  return p;
}

}  // namespace

fp8q_status moe_plan_quant_small(const void* x, int64_t T, int64_t H, int64_t ldx, const int* ids, int topk, int E,
                                 int format, const float* gscale, int* offsets, int* sf_offsets, int* pos, int* sf_row,
                                 void* q, uint8_t* sf, cudaStream_t stream) {
  Fp4QuantParams p = quant_params(x, T, H, ldx, format, gscale, q, H / 2, sf);
  p.topk = topk;
  const int wide = aligned(x, 32) && ldx % 16 == 0;
  return launch_kernel(format == FP8Q_FP4_NV ? moe_small_kernel<kNv> : moe_small_kernel<kMx>,
                       dim3(static_cast<unsigned>(T)), dim3(kItemThreads), 0, stream, 1, p, ids, E, offsets, sf_offsets,
                       pos, sf_row, wide);
}

}  // namespace fp8q

using namespace fp8q;

extern "C" size_t fp8q_fp4_sf_bytes(int64_t rows, int64_t K, int format) {
  if (rows <= 0 || K <= 0 || (format != FP8Q_FP4_NV && format != FP8Q_FP4_MX)) return 0;
  return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>(fp4_kblocks(format, K)) * 512;
}

extern "C" fp8q_status fp8q_fp4_quant(const void* x, int64_t M, int64_t K, int64_t ldx, int format,
                                      const float* gscale, void* q, int64_t ldq, uint8_t* sf, void* stream) {
  bool go;
  const fp8q_status st = check_quant(x, M, K, K, ldx, format, gscale, q, ldq, sf, &go);
  if (!go) return st;
  const Fp4QuantParams p = quant_params(x, M, K, ldx, format, gscale, q, ldq, sf);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? launch_items<kNv, OP_PLAIN>(p, s) : launch_items<kMx, OP_PLAIN>(p, s);
}

extern "C" fp8q_status fp8q_silu_mul_fp4_quant(const void* x, int64_t M, int64_t I, int64_t ldx, int format,
                                               const float* gscale, void* q, int64_t ldq, uint8_t* sf, void* stream) {
  bool go;
  const fp8q_status st = check_quant(x, M, I, 2 * I, ldx, format, gscale, q, ldq, sf, &go);
  if (!go) return st;
  const Fp4QuantParams p = quant_params(x, M, I, ldx, format, gscale, q, ldq, sf);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? launch_items<kNv, OP_SILU>(p, s) : launch_items<kMx, OP_SILU>(p, s);
}

extern "C" fp8q_status fp8q_rmsnorm_fp4_quant(const void* x, const void* w, float eps, int64_t M, int64_t H,
                                              int64_t ldx, int format, const float* gscale, void* q, int64_t ldq,
                                              uint8_t* sf, void* stream) {
  if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8Q_ERR_INVALID_ARG;
  bool go;
  const fp8q_status st = check_quant(x, M, H, H, ldx, format, gscale, q, ldq, sf, &go);
  if (!go) return st;
  if (!w || !aligned(w, 16)) return FP8Q_ERR_INVALID_ARG;
  Fp4QuantParams p = quant_params(x, M, H, ldx, format, gscale, q, ldq, sf);
  p.w = static_cast<const uint16_t*>(w);
  p.eps = eps;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? launch_rms<kNv>(p, s) : launch_rms<kMx>(p, s);
}

extern "C" fp8q_status fp8q_moe_fp4_quant(const void* x, int64_t T, int64_t K, int64_t ldx, int topk, const int* pos,
                                          const int* sf_row, int format, const float* gscale, void* q, int64_t ldq,
                                          uint8_t* sf, void* stream) {
  if (topk <= 0) return FP8Q_ERR_INVALID_ARG;
  bool go;
  const fp8q_status st = check_quant(x, T, K, K, ldx, format, gscale, q, ldq, sf, &go);
  if (!go) return st;
  if (!pos || !sf_row || !aligned(pos, 4) || !aligned(sf_row, 4)) return FP8Q_ERR_INVALID_ARG;
  Fp4QuantParams p = quant_params(x, T, K, ldx, format, gscale, q, ldq, sf);
  p.pos = pos;
  p.sf_row = sf_row;
  p.topk = topk;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? launch_items<kNv, OP_PLAIN>(p, s) : launch_items<kMx, OP_PLAIN>(p, s);
}

extern "C" fp8q_status fp8q_fp4_dequant(const void* q, int64_t ldq, const uint8_t* sf, int format,
                                        const float* gscale, int64_t M, int64_t K, void* y, int64_t ldy,
                                        void* stream) {
  if (format != FP8Q_FP4_NV && format != FP8Q_FP4_MX) return FP8Q_ERR_INVALID_ARG;
  if (M < 0 || K <= 0 || K % 32 != 0 || K > (int64_t{1} << 30) || M >= (int64_t{1} << 31)) return FP8Q_ERR_INVALID_ARG;
  if (ldq < K / 2 || ldq % 8 != 0 || ldy < K || ldy % 8 != 0) return FP8Q_ERR_INVALID_ARG;
  if (format == FP8Q_FP4_MX && gscale) return FP8Q_ERR_INVALID_ARG;
  if (M == 0) return FP8Q_OK;
  if (!q || !sf || !y || !aligned(q, 16) || !aligned(sf, 16) || !aligned(y, 16) || !aligned(gscale, 4))
    return FP8Q_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto kern = format == FP8Q_FP4_NV ? fp4_dequant_kernel<kNv> : fp4_dequant_kernel<kMx>;
  const int wide = aligned(y, 32) && ldy % 16 == 0;
  return launch_kernel(kern, dim3(item_blocks(M * (K >> 4))), dim3(kItemThreads), 0, s, 1,
                       static_cast<const uint8_t*>(q), ldq, sf, fp4_kblocks(format, K), gscale, M, K,
                       static_cast<uint16_t*>(y), ldy, wide);
}
