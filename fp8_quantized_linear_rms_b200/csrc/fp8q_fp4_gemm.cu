// fp8q_fp4_gemm.cu -- block-scaled products of 4-bit microscaled operands
// (nvfp4, mxfp4) on the tensor cores, dense and grouped by expert, bf16 out or
// with the experts' SiLU*mul and its requantization in the epilogue.
//
//   y[m, n] = bf16_rn( ga gb sum_k (qa[m, k] sfa[m, k/g]) (qb[n, k] sfb[n, k/g]) )
//
// The tensor core applies the scales (tcgen05.mma kind::mxf4nvf4 with four
// e4m3 scales per 64-deep K slice, kind::mxf4 with two E8M0), so the fp32
// accumulator stays in tensor memory for the whole K range.  Persistent CTAs,
// warp-specialized as in the FP8 GEMMs: warp 0 feeds a ring of stages (256
// codes = 128 bytes of every operand row, 128-byte swizzle by TMA, and the
// matching 512-byte scale blocks by plain bulk copies, which is why scales are
// stored in blocks), warp 1 copies a stage's scale blocks into tensor memory
// (tcgen05.cp) and issues its MMAs, the other warps are the epilogue.
//
// Tokens sit in the MMA's 128 rows, weights in its BN columns, at every size.
// A tile of few tokens copies only the 16- or 32-row pieces that hold some;
// the MMA then computes rows that nobody reads, at no cost where the time is
// that of reading the weights.  Where 128-row tiles do not fill the SMs (few
// tokens), a cluster of up to eight CTAs, two to an SM, splits the depth of a
// tile: each sums its part, and they add the parts over distributed shared
// memory in a fixed order.  (Narrower tiles instead: a 64-column MMA takes 59
// cycles, a 128-column one 65, so a stage of half the weights took as long.)
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "fp8q_common.cuh"
#include "fp8q_fp4_math.cuh"
#include "fp8q_sm100.cuh"

namespace fp8q {
namespace {

using namespace sm100;

constexpr int kStageBytes = 128;          // of an operand row: 256 codes
constexpr int kMaxExperts = 512;

struct Fp4Args {
  int64_t M, N, K;             // tokens (rows of all experts), weight rows of an expert, depth
  const uint8_t* sft;          // token scale blocks
  const uint8_t* sfw;          // weight scale blocks
  int kb;                      // scale blocks in a block row
  int kstages;                 // 256-deep steps
  int64_t wblocks;             // block rows of an expert's weight scales
  const float* ga;             // scale of the tokens' tensor (1 value) or null
  const float* gb;             // scales of the weights (one an expert) or null
  uint16_t* y;                 // bf16 [M, N] (not FUSED)
  int64_t ldy;
  const int* offsets;          // [E + 1] first row of each expert; null: dense
  const int* sf_offsets;       // [E + 1] first scale block row of each expert
  int E;
  uint8_t* hq;                 // FUSED: codes [M, I / 2], scale blocks, their tensor scale
  uint8_t* hsf;
  const float* gh;
  int64_t I;
  int tiles_n;                 // weight tiles of an expert
  int box;                     // token rows of one copy (16, 32, 128)
  int stages, ring;            // stages of the ring, and its bytes (a split tile's part lies there too)
  int a_bytes;                 // shared memory of a stage's token tile
  int split;                   // CTAs that share a tile's depth
  int share;                   // which rows of an expert: kAll, kPairs or kRest
  int* status;
};

// Experts' rows shared out between two launches: whole pairs of 128-row tiles
// (the last may lack some of its second), and a remainder of at most 128 rows.
constexpr int kAll = 0, kPairs = 1, kRest = 2;

// One lane of a converged warp.  The TMA and tcgen05 instructions take uniform
// registers; in code under elect.sync the compiler knows that one lane runs and
// issues them directly, while under `lane == 0` it wraps each in a loop over
// the warp's active lanes (measured: 64 against 18 cycles a tcgen05.cp, 109
// against 59 a 64-column MMA).  The loops around it are run by the whole warp,
// so that addresses and descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= (A SFA)(B SFB)^T, both e2m1.
#define FP4_MMA(GROUP, KIND)                                                                                    \
  asm volatile(                                                                                                 \
      "{\n\t.reg .pred p;\n\t"                                                                                  \
      "setp.ne.b32 p, %4, 0;\n\t"                                                                               \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d), "l"(a),  \
      "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)                                                          \
      : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                        uint32_t sfa, uint32_t sfb) {
  if constexpr (FMT == kNv) {
    if constexpr (PAIR) FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if constexpr (PAIR) FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  }
}
#undef FP4_MMA

// Arrive on the even CTA's barrier without releasing memory: what the MMAs wait
// for is that tensor memory has been read, which tcgen05.wait::ld and the
// tcgen05 fence order; a release at cluster scope would also wait for this
// thread's stores to y (~1300 cycles a tile).
__device__ __forceinline__ void arrive_relaxed(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// Whether a barrier's phase is complete, without waiting: test_wait, since
// try_wait suspends the warp for microseconds when it is not.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A 512-byte scale block -- 32 rows of 16 bytes, row l the scales of operand
// rows l, l + 32, l + 64, l + 96 -- from shared memory into 4 columns of all
// four lane quadrants of tensor memory (of both CTAs, each from its own shared
// memory, for a pair).  Descriptor: K-major, no swizzle, 8-row core matrices
// 128 bytes apart, version 1.  A thread's copies and MMAs run in issue order.
__device__ __forceinline__ uint64_t scales_desc(const void* src) {
  return (static_cast<uint64_t>(smem_u32(src) & 0x3FFFF) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t col, uint64_t desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(col), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(col), "l"(desc) : "memory");
}

// Instruction descriptor of the 4-bit block-scaled kinds: scale id of B (bits
// 4-5) and A (29-30), e2m1 operands (bits 7-9 and 10-12 = 1), K-major, N >> 3
// at bits 17-22, scale format (bit 23: 0 e4m3, 1 E8M0), M >> 7 at bits 27-28.
__device__ __forceinline__ uint32_t idesc_fp4(int fmt, int M, int N, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(fmt == kMx) << 23) | (static_cast<uint32_t>(M >> 7) << 27) | (id << 29);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A value that all lanes of the warp hold, in a uniform register: what comes
// from shared memory the compiler must take for different in every lane, and
// then every address and loop that depends on it too.  A warp reduction's
// result it knows to be uniform.  (A stage's two copies took ~430 cycles to
// issue without it.)
__device__ __forceinline__ int uniform(int v) {
  return static_cast<int>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(v)));
}

// A tile: its expert, first token row and how many rows are the expert's, the
// token scales' block row, and the first weight row (of the expert).
struct Fp4Tile {
  int e, t0, cnt, tblk, n0;
};

// What a CTA keeps of an expert in shared memory (read once, so that a tile
// costs no loads from global memory): token tiles before it, its first row,
// its rows, and the first block row of its scales.
struct Fp4Expert {
  int tiles, first, rows, sf;
};

// Tile u (the whole warp calls): an expert's tiles are consecutive, its token
// tiles the fastest index (they share the weight tile, which then comes from
// L2).  A CTA pair's tile has 256 token rows; `rank` says which 128 of them.
template <bool PAIR>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4Args& p, const Fp4Expert* ex, int u, int tn, int rank) {
  constexpr int TM = PAIR ? 256 : 128;
  int lo = 0;
  if (p.E > 1) {
    // the last expert with no more than u tiles before it, in steps of 32 and of 1
    const int lane = threadIdx.x & 31, step = (p.E + 31) >> 5;
    const int e = lane * step;
    lo = (__popc(__ballot_sync(0xFFFFFFFFu, e < p.E && ex[e < p.E ? e : 0].tiles * p.tiles_n <= u)) - 1) * step;
    const int f = lo + lane;
    const bool in = lane < step && f < p.E;
    lo += __popc(__ballot_sync(0xFFFFFFFFu, in && ex[in ? f : 0].tiles * p.tiles_n <= u)) - 1;
  }
  lo = uniform(lo);
  const Fp4Expert x = {uniform(ex[lo].tiles), uniform(ex[lo].first), uniform(ex[lo].rows), uniform(ex[lo].sf)};
  const int mt = (x.rows + TM - 1) / TM;
  const int r = u - x.tiles * p.tiles_n;
  const int nt = mt == 1 ? r : uniform(r / mt), m = r - nt * mt;
  const int b = PAIR ? 2 * m + rank : m;
  Fp4Tile t;
  t.e = lo;
  t.t0 = x.first + 128 * b;
  t.cnt = max(0, min(128, x.rows - 128 * b));
  t.tblk = x.sf + b;
  t.n0 = nt * tn;
  return t;
}

// ------------------------------------------------------------------- kernel
// CH output columns a tile: 128 or 256 weight rows, or FUSED 128 hidden
// channels, whose 128 gate rows are followed by the up rows.
// PAIR: two CTAs of a cluster share one MMA of 256 token rows and 256 columns
// (tcgen05 cta_group::2), each with 128 of the rows of both operands in its
// shared memory, so a weight row reaches each SM half as often; each holds the
// scales of its own tokens and of all columns.  Tried and slower: a tile as two
// 128-column MMAs and accumulators, so that one is read while the other
// computes (a pair's 128-column MMA took ~140 cycles, more than the 256-column
// one: 1341 against 894 us at 8192 x 51200 x 5120).
// SPLIT: one tile of 128 weight rows a cluster, whose CTAs share its depth;
// FUSED, half of them take the gate rows and half the up rows.
template <int FMT, int CH, bool FUSED, bool PAIR, bool SPLIT>
struct Fp4Cfg {
  static constexpr int PER_SM = SPLIT ? 2 : 1;              // CTAs on an SM, by tensor memory
  static constexpr int HALVES = SPLIT && FUSED ? 2 : 1;     // CTAs for gate and up
  static constexpr int BN = FUSED ? 2 * CH / HALVES : CH;   // accumulator columns
  static constexpr int EPI_WARPS = SPLIT ? 4 : 8;
  static constexpr int THREADS = 96 + 32 * EPI_WARPS;
  static constexpr int NKB = FMT == kNv ? 4 : 2;            // scale blocks of a stage, per 128 rows
  static constexpr int SF_BYTES = NKB * 512;                // per 128 rows
  static constexpr int SF_COLS = NKB * 4;
  static constexpr int BBLK = BN / 128;                     // 128-row blocks of weight rows
  static constexpr int B_BYTES = (PAIR ? 128 : BN) * kStageBytes;
  static constexpr int SF_STAGE = (1 + BBLK) * SF_BYTES;
  static constexpr int SF_TMEM = (1 + BBLK) * SF_COLS;      // tensor memory columns of a stage's scales
  static constexpr int SFBUF = SPLIT ? 1 : 4;               // stages' scales in tensor memory at once
  static constexpr int NBUF = BN == 256 || SPLIT ? 1 : 2;   // accumulators
  static constexpr int ACC_COLS = NBUF * BN;
  static constexpr int TMEM = 512 / PER_SM;
  static constexpr bool STAGED = !FUSED && !SPLIT;          // y leaves through shared memory
  static constexpr int OUT_BYTES = STAGED ? EPI_WARPS * 4096 : 0;
  static_assert(ACC_COLS + SFBUF * SF_TMEM <= TMEM, "tensor memory");
  static_assert(!PAIR || (BN == 256 && !SPLIT && !FUSED), "pairs: 256 columns");
  static_assert(!SPLIT || BN == 128, "split tiles have 128 columns");
};

template <int FMT, int CH, bool FUSED, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(Fp4Cfg<FMT, CH, FUSED, PAIR, SPLIT>::THREADS,
                                  Fp4Cfg<FMT, CH, FUSED, PAIR, SPLIT>::PER_SM)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmTS, const __grid_constant__ CUtensorMap tmWS,
                    const Fp4Args p) {
  using C = Fp4Cfg<FMT, CH, FUSED, PAIR, SPLIT>;
  constexpr int BN = C::BN, NB = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = p.stages;
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * p.a_bytes;
  uint8_t* sSF = sB + S * C::B_BYTES;
  uint8_t* sOut = smem + p.ring;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + C::OUT_BYTES);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = full + 30;        // 16-byte aligned, whatever S <= 12
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* all_tiles = reinterpret_cast<int*>(tmem_slot + 2);
  Fp4Expert* ex = reinterpret_cast<Fp4Expert*>(drain + 4);              // [E]

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  // the tile loop: first tile and step; SPLIT: one tile, of whose depth this
  // CTA takes stages [k0, k1), of the gate or the up rows (half)
  const int group = SPLIT ? p.split * C::HALVES : PAIR ? 2 : 1;
  const int cta = uniform(static_cast<int>(blockIdx.x) / group), ctas = uniform(static_cast<int>(gridDim.x) / group);
  const int part = SPLIT ? static_cast<int>(blockIdx.x) - cta * group : 0;
  const int half = C::HALVES == 2 && part >= p.split ? 1 : 0, kpart = part - half * p.split;
  const int k0 = SPLIT ? uniform(p.kstages * kpart / p.split) : 0;
  const int k1 = SPLIT ? uniform(p.kstages * (kpart + 1) / p.split) : p.kstages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::EPI_WARPS * (PAIR ? 2 : 1));
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmT);
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, C::TMEM);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM);
      tmem_relinquish();
    }
  }
  if (warp == 0 && p.offsets == nullptr && cta < (p.M + 127) / 128 * p.tiles_n) {
    // The first stages' weights into L2 while the previous kernel of the stream
    // finishes: a hint (they are loaded again after the wait).
    const int64_t tm = (p.M + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128);
    const int n0 = static_cast<int>(cta / tm) * CH + (PAIR ? rank * 128 : 0);
    if (elect_one()) {
      for (int kb = k0; kb < k1 && kb < k0 + S; ++kb) {
        tma_prefetch_2d(&tmW, kb * kStageBytes, n0);
        if (C::BBLK == 2 && !PAIR) tma_prefetch_2d(&tmW, kb * kStageBytes, n0 + 128);
      }
    }
    __syncwarp();
  }
  // The rest's launch follows the pairs', which had waited for what both read
  // before it let this one start: it waits for the pairs themselves at its end,
  // and takes the SMs that they leave one by one.  (Plain loads go to L2, past
  // what an L1 may hold of an earlier call's.)
  if (p.share != kRest) griddep_wait();

  constexpr int kTM = PAIR ? 256 : 128;
  if (p.offsets == nullptr) {
    if (threadIdx.x == 0) {
      ex[0] = {0, 0, static_cast<int>(p.M), 0};
      *all_tiles = static_cast<int>((p.M + kTM - 1) / kTM);
    }
  } else {
    for (int e = threadIdx.x; e < p.E; e += C::THREADS) {
      // whatever the arrays hold, rows stay below M and scales inside their buffer
      const int M = static_cast<int>(p.M), first = min(max(__ldcg(p.offsets + e), 0), M);
      const int rows = min(max(__ldcg(p.offsets + e + 1), first), M) - first;
      const int most = M / 128 + min(M, p.E) - (rows + 127) / 128;
      Fp4Expert x = {0, first, rows, min(max(__ldcg(p.sf_offsets + e), 0), most)};
      if (p.share != kAll) {
        const int rest = (rows & 255) <= 128 ? rows & 255 : 0;
        if (p.share == kPairs) x.rows -= rest;
        else x = {0, first + rows - rest, rest, x.sf + (rows - rest) / 128};
      }
      ex[e] = x;
    }
    __syncthreads();
    if (warp == 0) {
      int carry = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const int tiles = e < p.E ? (ex[e].rows + kTM - 1) / kTM : 0;
        int v = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int w = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += w;
        }
        if (e < p.E) ex[e].tiles = carry + v - tiles;
        carry += __shfl_sync(0xFFFFFFFFu, v, 31);
      }
      if (lane == 0) *all_tiles = carry;
    }
  }
  tc_fence_before();
  __syncthreads();
  griddep_launch_dependents();             // this CTA has its tensor memory: a dependent cannot take it first
  if constexpr (PAIR) cluster_sync();      // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  const int units = uniform(*all_tiles) * p.tiles_n;

  // SPLIT: the tile, and the factors that its output takes, before the long wait
  Fp4Tile tile0{};
  const Fp4G gh = fp4_g(FUSED ? p.gh : nullptr);
  const float ga = p.ga ? __ldcg(p.ga) : 1.0f;
  float gb = 1.0f;
  if (SPLIT && cta < units) {
    tile0 = fp4_tile<PAIR>(p, ex, cta, CH, 0);
    if (p.gb) gb = __ldcg(p.gb + tile0.e);
  }
  // a wait by the whole warp; false in all lanes if one gave up
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status)) != 0;
  };

  if (warp == 0 || warp == 2 + C::EPI_WARPS) {
    // ------------------------------------------------------------ producers
    // One warp copies weights and their scales, another the tokens' (four
    // copies a stage by one warp took as long as the stage's MMAs).  The first
    // announces a stage's bytes; the barrier cannot complete before it does.
    const bool tokens = warp != 0;
    int it = 0, st = 0;
    uint32_t parity = 1;
    bool ok = true;
    for (int u = cta; ok && u < units; u += ctas) {
      const Fp4Tile t = fp4_tile<PAIR>(p, ex, u, CH, rank);
      const int up = FUSED ? static_cast<int>(p.I) : 128;       // from the first 128 weight rows to the second
      const int wrow = t.e * static_cast<int>(p.N) + t.n0 + (PAIR ? rank : half) * up;
      const int pieces = (t.cnt + p.box - 1) / p.box;
      const int64_t wblk = t.e * p.wblocks + ((t.n0 + half * up) >> 7);
      const uint8_t* sft = p.sft + static_cast<int64_t>(t.tblk) * p.kb * 512;
      const uint8_t* sfw = p.sfw + wblk * p.kb * 512;
      // a second block of weight scales: the up half's, or columns 128..255
      const int64_t second = static_cast<int64_t>(up >> 7) * p.kb * 512;
      const bool two = C::BBLK == 2 && (FUSED || t.n0 + 128 < p.N);
      // bytes of a stage beside the scales: of both CTAs of a pair, whose boxes count in full
      int bytes = pieces * p.box * kStageBytes + C::B_BYTES;
      if constexpr (PAIR) {
        const int other = fp4_tile<PAIR>(p, ex, u, CH, 1).cnt;
        bytes += (other + p.box - 1) / p.box * p.box * kStageBytes + C::B_BYTES + 6 * C::SF_BYTES;
      }
      bool ready = mbar_test(&empty[st], parity);
      for (int kb = k0; kb < k1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, ready) && !warp_wait(&empty[st], parity)) { ok = false; break; }
        const int cur = st;
        ++it;
        if (++st == S) { st = 0; parity ^= 1u; }
        ready = mbar_test(&empty[st], parity);              // the next stage's, while this one is issued
        uint8_t* a = sA + cur * p.a_bytes;
        uint8_t* b = sB + cur * C::B_BYTES;
        uint8_t* s = sSF + cur * C::SF_STAGE;
        const int x = kb * kStageBytes;
        const uint32_t sfb = min(C::NKB, p.kb - kb * C::NKB) * 512;
        const int64_t sfo = static_cast<int64_t>(kb) * C::SF_BYTES;
        if (elect_one()) {
          if constexpr (PAIR) {
            // everything lands on the even CTA's barrier
            const uint32_t bar = mapa_shared(smem_u32(&full[cur]), 0);
            const int y = kb * C::NKB;
            if (!tokens) {
              if (rank == 0) mbar_arrive_expect_tx(&full[cur], bytes);
              tma_load_2d_pair(b, &tmW, bar, x, wrow);
              tma_load_2d_pair(s + C::SF_BYTES, &tmWS, bar, 0, static_cast<int>(wblk) * p.kb + y);
              tma_load_2d_pair(s + 2 * C::SF_BYTES, &tmWS, bar, 0, static_cast<int>(wblk + (up >> 7)) * p.kb + y);
            } else {
              for (int i = 0; i < pieces; ++i)
                tma_load_2d_pair(a + i * p.box * kStageBytes, &tmT, bar, x, t.t0 + i * p.box);
              tma_load_2d_pair(s, &tmTS, bar, 0, t.tblk * p.kb + y);
            }
          } else if (!tokens) {
            mbar_arrive_expect_tx(&full[cur], bytes + (two ? 3 : 2) * sfb);
            tma_load_2d(b, &tmW, &full[cur], x, wrow);
            if (C::BBLK == 2) tma_load_2d(b + 128 * kStageBytes, &tmW, &full[cur], x, wrow + up);
            bulk_load(s + C::SF_BYTES, sfw + sfo, sfb, &full[cur]);
            if (two) bulk_load(s + 2 * C::SF_BYTES, sfw + second + sfo, sfb, &full[cur]);
          } else {
            for (int i = 0; i < pieces; ++i)
              tma_load_2d(a + i * p.box * kStageBytes, &tmT, &full[cur], x, t.t0 + i * p.box);
            bulk_load(s, sft + sfo, sfb, &full[cur]);
          }
        }
        __syncwarp();
      }
    }
    // Let the copies in flight land before this CTA (or its pair) can leave; at
    // once when everything was consumed.
    const int first = it - S > 0 ? it - S : 0;
    for (int j = first; (PAIR ? rank == 0 : !ok) && j < it; ++j) drain_wait(&full[j % S], (j / S) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the even CTA's, of a pair)
    if (rank == 0) {
      const uint32_t id0 = idesc_fp4(FMT, PAIR ? 256 : 128, BN, 0);
      auto commit = [](uint64_t* bar) {
        if constexpr (PAIR) mma_commit_pair(bar, 0x3);
        else mma_commit(bar);
      };
      const uint64_t a_desc = smem_desc_kmajor_sw128(sA), b_desc = smem_desc_kmajor_sw128(sB);
      const uint64_t sf_desc = scales_desc(sSF);
      int st = 0, sbuf = 0, buf = 0;
      uint32_t parity = 0, acc_parity = 1;
      bool ok = true;
      for (int u = cta; ok && u < units; u += ctas) {
        if (!warp_wait(&tempty[buf], acc_parity)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        bool ready = mbar_test(&full[st], parity);
        for (int kb = k0; kb < k1; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, ready) && !warp_wait(&full[st], parity)) { ok = false; break; }
          tc_fence_after();
          const int cur = st;
          if (++st == S) { st = 0; parity ^= 1u; }
          ready = mbar_test(&full[st], parity);             // the next stage's, while this one is issued
          const uint32_t sfa = tmem + C::ACC_COLS + sbuf * C::SF_TMEM;
          const uint32_t sfb = sfa + C::SF_COLS;
          const uint64_t sd = sf_desc + static_cast<uint32_t>(cur * (C::SF_STAGE >> 4));
          const uint64_t ad = a_desc + static_cast<uint32_t>(cur * (p.a_bytes >> 4));
          const uint64_t bd = b_desc + static_cast<uint32_t>(cur * (C::B_BYTES >> 4));
          const int nk = p.kb - kb * C::NKB;                       // scale blocks and K slices left
          const int ks = static_cast<int>((p.K - static_cast<int64_t>(kb) * 256 + 63) >> 6);
          if (elect_one()) {
#pragma unroll
            for (int b = 0; b < C::NKB; ++b) {
              if (b < nk) {
                cp_scales<PAIR>(sfa + b * 4, sd + (b * 512 >> 4));
#pragma unroll
                for (int j = 0; j < C::BBLK; ++j)
                  cp_scales<PAIR>(sfb + b * (4 * C::BBLK) + j * 4, sd + (((1 + j) * C::SF_BYTES + b * 512) >> 4));
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k < ks) {
                // nvfp4: a K slice has a scale block of its own; mxfp4: two share one, ids 0 and 2
                const int b = FMT == kNv ? k : k >> 1;
                const uint32_t id = FMT == kNv ? 0u : 2u * (k & 1);
                mma_fp4<FMT, PAIR>(d, ad + 2 * k, bd + 2 * k, id0 | (id << 4) | (id << 29), kb > k0 || k > 0,
                                   (sfa + b * 4) | (id << 30), (sfb + b * (4 * C::BBLK)) | (id << 30));
              }
            }
            commit(&empty[cur]);
            if (kb + 1 == k1) commit(&tfull[buf]);
          }
          __syncwarp();
          if (++sbuf == C::SFBUF) sbuf = 0;
        }
        if (++buf == NB) { buf = 0; acc_parity ^= 1u; }
      }
      // every MMA issued has completed once `drain` flips
      if (elect_one()) commit(drain);
      __syncwarp();
    }
    drain_wait(drain, 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;                        // tensor memory lanes 32 quad ..
    const int r = quad * 32 + lane;                   // this thread's token of the tile
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    constexpr int COLS = CH / (C::EPI_WARPS / 4);     // output columns of a thread (not SPLIT)
    const int col0 = ((warp - 2) >> 2) * COLS;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : 0u;
    // the accumulator goes back to the MMAs (of the even CTA)
    auto give_back = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) arrive_relaxed(tempty0 + 8u * buf);
        else mbar_arrive(&tempty[buf]);
      }
    };
    int buf = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int u = cta; ok && u < units; u += ctas) {
      const Fp4Tile t = SPLIT ? tile0 : fp4_tile<PAIR>(p, ex, u, CH, rank);
      if (!SPLIT && p.gb) gb = __ldcg(p.gb + t.e);      // on its way while the tile is computed
      if constexpr (SPLIT) {
        // This CTA's part of the tile, fp32, over the ring (whose copies and MMAs
        // are done): row r at r BN, 16-byte chunks XORed by the row.
        if (!warp_wait(&tfull[0], parity)) { ok = false; break; }
        tc_fence_after();
        constexpr int PART = BN / (C::EPI_WARPS / 4);
        if (quad * 32 < t.cnt) {
#pragma unroll 1
          for (int c = 0; c < PART; c += 32) {
            const int col = ((warp - 2) >> 2) * PART + c;
            uint32_t v[32];
            tmem_ld_waited<32>(tmem + lane_addr + col, v);
            uint4* d = reinterpret_cast<uint4*>(smem + r * (BN * 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              d[(col / 4 + i) ^ (r & 7)] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      } else if constexpr (!FUSED) {
        if (!warp_wait(&tfull[buf], parity)) { ok = false; break; }
        const float alpha = ga * gb;
        tc_fence_after();
        // The thread's columns, rounded to bf16 as they are read (the next 32 in
        // flight meanwhile), so that the accumulator goes back to the MMAs
        // before anything is stored.
        uint32_t o[COLS / 2];
        if (quad * 32 < t.cnt) {
          const uint32_t acc = tmem + lane_addr + buf * BN + col0;
          uint32_t v[2][32];
          tmem_ld_async<32>(acc, v[0]);
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            uint32_t* w = v[(c / 32) & 1];
            tmem_wait_regs<32>(w);
            if (c + 32 < COLS) tmem_ld_async<32>(acc + c + 32, v[(c / 32 + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              o[(c + i) / 2] = pack_bf16(__uint_as_float(w[i]) * alpha, __uint_as_float(w[i + 1]) * alpha);
          }
        }
        give_back(buf);
        if (++buf == NB) { buf = 0; parity ^= 1u; }
        const int64_t n = t.n0 + col0;
        {
          // A lane's row of 64 columns (128 bytes) through shared memory, 16-byte
          // chunks XORed by the row, so that eight lanes store a whole line of y:
          // stored from the lane that holds it, a 32-byte piece costs a line's
          // transaction (a 128 x 256 tile's stores took ~5000 cycles).
          uint8_t* mine = sOut + (warp - 2) * 4096;
#pragma unroll
          for (int c = 0; c < COLS / 2; c += 32) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(mine + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_uint4(o[c + 4 * i], o[c + 4 * i + 1], o[c + 4 * i + 2], o[c + 4 * i + 3]);
            __syncwarp();
            const int64_t col = n + 2 * c + 8 * (lane & 7);
            uint16_t* y = p.y + static_cast<int64_t>(t.t0 + quad * 32) * p.ldy + col;
            if (col < p.N) {
#pragma unroll
              for (int i = lane >> 3; i < 32; i += 4)
                if (quad * 32 + i < t.cnt)
                  *reinterpret_cast<uint4*>(y + i * p.ldy) =
                      *reinterpret_cast<const uint4*>(mine + i * 128 + (((lane ^ i) & 7) << 4));
            }
          }
        }
      } else {
        // The same gate and up columns of the thread's row; the accumulator
        // goes back once they are in registers.
        if (!warp_wait(&tfull[0], parity)) { ok = false; break; }
        const float alpha = ga * gb;
        parity ^= 1u;
        tc_fence_after();
        const uint32_t acc = tmem + lane_addr + col0;
        const int64_t n = t.n0 + col0;
        uint32_t g[COLS], w[COLS];
        if (quad * 32 < t.cnt) {
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            tmem_ld_async<32>(acc + c, g + c);
            tmem_ld_async<32>(acc + CH + c, w + c);
          }
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            tmem_wait_regs<32>(g + c);
            tmem_wait_regs<32>(w + c);
          }
        }
        give_back(0);
        if (r < t.cnt) {
          constexpr int G = fp4_group<FMT>();
          uint32_t code[COLS / 8], sfw = 0;
#pragma unroll
          for (int j = 0; j < COLS; j += G) {
            float y[G], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < G; ++i) {
              y[i] = silu_mul_f32(__uint_as_float(g[j + i]) * alpha, __uint_as_float(w[j + i]) * alpha);
              amax = fmaxf(amax, fabsf(y[i]));
            }
            const Fp4Scale s = fp4_scale<FMT>(amax, gh);
            sfw |= s.byte << (8 * (j / G));
#pragma unroll
            for (int i = 0; i < G; i += 8) code[(j + i) / 8] = fp4_codes8<FMT>(y + i, s);
            if (fp4_far<FMT>(amax, s)) {
#pragma unroll
              for (int i = 0; i < G; i += 8) code[(j + i) / 8] = fp4_codes8_far(y + i, s);
            }
          }
          uint4* q = reinterpret_cast<uint4*>(p.hq + static_cast<int64_t>(t.t0 + r) * (p.I >> 1) + (n >> 1));
#pragma unroll
          for (int c = 0; c < COLS / 8; c += 4)
            q[c / 4] = make_uint4(code[c], code[c + 1], code[c + 2], code[c + 3]);
          // tiles begin at a block row of the scales; a thread's scales are aligned 1 to 4 bytes of a word
          uint8_t* sf = p.hsf + fp4_sf_offset(static_cast<int64_t>(t.tblk) * 128 + r, n / G, fp4_kblocks(FMT, p.I));
          if constexpr (COLS / G == 4) *reinterpret_cast<uint32_t*>(sf) = sfw;
          else if constexpr (COLS / G == 2) *reinterpret_cast<uint16_t*>(sf) = static_cast<uint16_t>(sfw);
          else *sf = static_cast<uint8_t>(sfw);
        }
      }
    }
  }

  if constexpr (SPLIT) {
    // The parts of the cluster's CTAs, added in the order of the depth.  Its
    // warps take turns at pieces of a row: 32 hidden channels, a lane each, or
    // 32 chunks of 8 outputs (two rows, one, or part of one).
    cluster_sync();
    if (cta < units && *abort_flag == 0) {
      const Fp4Tile& t = tile0;
      const float alpha = ga * gb;
      constexpr int WARPS = C::THREADS / 32, UNIT = FUSED ? 1 : 8, PIECES = CH / UNIT;   // of a row
      for (int i0 = (part * WARPS + warp) * 32; i0 < t.cnt * PIECES; i0 += group * WARPS * 32) {
        const int row = (i0 + lane) / PIECES, col = (i0 + lane - row * PIECES) * UNIT;
        float v[FUSED ? 2 : 8] = {};
        if (row < t.cnt) {
          for (int q = 0; q < p.split; ++q) {
            const uint32_t src = mapa_shared(smem_u32(smem), q) + row * (BN * 4);
            const uint32_t at = src + (((col >> 2) ^ (row & 7)) << 4);
            if constexpr (FUSED) {
              float g, u;
              asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(g) : "r"(at + 4 * (col & 3)) : "memory");
              const uint32_t upper = mapa_shared(smem_u32(smem), p.split + q) + (at - mapa_shared(smem_u32(smem), q));
              asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(upper + 4 * (col & 3)) : "memory");
              v[0] += g;
              v[1] += u;
            } else {
              float f[8];
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(at) : "memory");
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                           : "r"(src + ((((col >> 2) + 1) ^ (row & 7)) << 4)) : "memory");
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] += f[k];
            }
          }
        }
        const int64_t n = t.n0 + col;
        if constexpr (FUSED) {
          // whole warps: the channels of a row are four warps' worth
          constexpr int G = fp4_group<FMT>();
          const float y = silu_mul_f32(v[0] * alpha, v[1] * alpha);
          float amax = fabsf(y);
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          const Fp4Scale sc = fp4_scale<FMT>(amax, gh);
          uint32_t code = fp4_code1<FMT>(y, sc) << (4 * (lane & 7));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) code |= __shfl_xor_sync(0xFFFFFFFFu, code, o);
          if ((lane & 7) == 0)
            *reinterpret_cast<uint32_t*>(p.hq + static_cast<int64_t>(t.t0 + row) * (p.I >> 1) + (n >> 1)) = code;
          if (lane % G == 0)
            p.hsf[fp4_sf_offset(static_cast<int64_t>(t.tblk) * 128 + row, n / G, fp4_kblocks(FMT, p.I))] =
                static_cast<uint8_t>(sc.byte);
        } else if (row < t.cnt && n < p.N) {
          *reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(t.t0 + row) * p.ldy + n) =
              make_uint4(pack_bf16(v[0] * alpha, v[1] * alpha), pack_bf16(v[2] * alpha, v[3] * alpha),
                         pack_bf16(v[4] * alpha, v[5] * alpha), pack_bf16(v[6] * alpha, v[7] * alpha));
        }
      }
    }
    cluster_sync();                          // no part is given up while another CTA reads it
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();      // neither leaves while the other may use its memory
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, C::TMEM);
    else tmem_dealloc(tmem, C::TMEM);
  }
  if (p.share == kRest) griddep_wait();
}

// ------------------------------------------------------------------ host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Codes [rows, K / 2] bytes, box = box_rows x 128 bytes, 128-byte swizzle,
// zero (code 0) outside the matrix.
bool fp4_tensor_map(const void* ptr, int64_t rows, int64_t K, int box_rows, CUtensorMap* out) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t gstride[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {kStageBytes, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estride[2] = {1, 1};
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale blocks as rows of 512 bytes; box = `rows` blocks.
bool fp4_scale_map(const void* ptr, int64_t blocks, int rows, CUtensorMap* out) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {128, static_cast<cuuint64_t>(blocks)};
  const cuuint64_t gstride[1] = {512};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(rows)};
  const cuuint32_t estride[2] = {1, 1};
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSmemMax = 227 * 1024;
constexpr int kSmemSm = 228 * 1024;     // of an SM; 1 KB of each CTA's share is reserved
constexpr int kBarBytes = 8 * 34;       // barriers, tensor memory address, abort flag, tile count

template <int FMT, int CH, bool FUSED, bool PAIR, bool SPLIT>
fp8q_status launch_fp4(const void* t, const void* w, int64_t tiles_t, Fp4Args& p, cudaStream_t stream) {
  using C = Fp4Cfg<FMT, CH, FUSED, PAIR, SPLIT>;
  CUtensorMap mt, mw, mts, mws;
  if (!fp4_tensor_map(t, p.M, p.K, p.box, &mt) || !fp4_tensor_map(w, p.E * p.N, p.K, 128, &mw))
    return FP8Q_ERR_CUDA;
  if (PAIR) {
    const int64_t tblocks = p.offsets ? p.M / 128 + (p.M < p.E ? p.M : p.E) : (p.M + 127) / 128;
    if (!fp4_scale_map(p.sft, tblocks * p.kb, C::NKB, &mts) ||
        !fp4_scale_map(p.sfw, p.E * p.wblocks * p.kb, C::NKB, &mws))
      return FP8Q_ERR_CUDA;
  } else {
    mts = mt;      // not read
    mws = mw;
  }
  p.tiles_n = static_cast<int>(((FUSED ? p.I : p.N) + CH - 1) / CH);
  // A tile that is known to have fewer rows keeps less of them; its MMA reads
  // 128 rows' worth of shared memory from the tile's start all the same.
  p.a_bytes = p.M <= 128 ? static_cast<int>((p.M + p.box - 1) / p.box) * p.box * kStageBytes : 128 * kStageBytes;
  const int stage = p.a_bytes + C::B_BYTES + C::SF_STAGE;
  const int fixed = 1024 + C::OUT_BYTES + kBarBytes + 16 * p.E;      // alignment, ...
  const int64_t units = tiles_t * p.tiles_n;
  auto stages = [&](int per_sm) {
    const int n = ((per_sm == 1 ? kSmemMax : kSmemSm / per_sm - 1024) - fixed) / stage;
    return n > 12 ? 12 : n;
  };
  int per_sm = 1, part = 0;
  p.split = 1;
  if (SPLIT) {
    // about one CTA an SM: a tile's depth in up to eight parts of two stages at
    // least.  (More and shorter parts were slower: 1 x 5120 x 25600 nvfp4 took
    // 18.1 us in 3 parts, 19.2 in 4; clusters that do not fit at once wait for
    // the first to end, so split tiles leave room for two CTAs on an SM.)
    p.split = static_cast<int>(units > 0 ? num_sms() / (units * C::HALVES) : 1);
    if (p.split > 8 / C::HALVES) p.split = 8 / C::HALVES;
    if (p.split > p.kstages / 2) p.split = p.kstages / 2;
    if (p.split < 1) p.split = 1;
    if (units * p.split * C::HALVES > num_sms() || p.split * C::HALVES > 1) per_sm = 2;
    part = (p.M < 128 ? static_cast<int>(p.M + 31) / 32 * 32 : 128) * C::BN * 4;
  }
  p.stages = stages(per_sm);
  p.ring = p.stages * stage;
  // the MMA's reach from the last stage's token tile, and a split tile's part
  const int reach = (p.stages - 1) * p.a_bytes + 128 * kStageBytes;
  if (p.ring < reach) p.ring = reach;
  if (p.ring < part) p.ring = part;
  int smem = fixed + p.ring;
  // No less shared memory than the CTA's share of tensor memory: CTAs that fit
  // an SM together then never wait for each other's tensor memory, which CTAs
  // of a cluster that wait for one another must not do.
  if (SPLIT && smem < kSmemSm / C::PER_SM - 1024) smem = kSmemSm / C::PER_SM - 1024;
  auto kern = fp4_gemm_kernel<FMT, CH, FUSED, PAIR, SPLIT>;
  static std::atomic<int> attr_done[64];     // CTAs (pairs) that fit the device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8Q_ERR_CUDA;
  int fit = attr_done[dev].load(std::memory_order_relaxed);
  if (!fit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    fit = num_sms();
    if (PAIR) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 * static_cast<unsigned>(num_sms()));
      cfg.blockDim = dim3(C::THREADS);
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess || fit < 1) return FP8Q_ERR_CUDA;
    }
    attr_done[dev].store(fit, std::memory_order_relaxed);
  }
  if (SPLIT)
    return launch_kernel(kern, dim3(static_cast<unsigned>(units * p.split * C::HALVES)), dim3(C::THREADS), smem, stream,
                         p.split * C::HALVES, mt, mw, mts, mws, p);
  const unsigned grid = static_cast<unsigned>(units < fit ? units : fit) * (PAIR ? 2 : 1);
  return launch_kernel(kern, dim3(grid), dim3(C::THREADS), smem, stream, PAIR ? 2 : 1, mt, mw, mts, mws, p);
}

// Variant and launch, by how many tiles there are for the SMs.  Measured on
// both sides of each border (us):
//   split tiles up to half as many 128-row tiles as SMs: 16 x 4096 x 12288
//     mxfp4 (32 tiles) 9.7 split, 18.5 not; 1 x 10240 x 5120 (80) 11.2 and 11.0
//   CTA pairs from as many 256 x 256 tiles as pairs of SMs: 512 x 10240 x 5120
//     nvfp4 (80) 22.2 in pairs, 25.0 with 128 rows, 25.5 with 256; 256 x 5120 x
//     5120 (20) 13, 10.6 and 12.9.  Experts' rows are ragged: pairs take the
//     whole tiles, and the remainders, in a launch of their own, the SMs that
//     the pairs leave.  Down products from 768 rows an expert on: 16 experts,
//     4096 outputs of depth 2048, 1024 rows 91 without, 82-87 in pairs, 2048
//     rows 224-230 and 149-160; 64, 2048 of 1408 mxfp4, 1024 rows 162-168 and
//     121-138; 128, 2048 of 768, 256 rows 55 and 60, 512 rows 88-96 and 96-99,
//     768 rows 188 and 159.  gate_up lost (256 rows 76 and 83) or drew
//   256 weight rows unless 128 spread over the SMs in less than twice as many
//     rounds: 1 x 51200 x 5120 (400 tiles of 128: 3 rounds, 200 of 256: 2) 29.4
//     with 256, 26.2 with 128; 1 x 24576 x 4096 (2 and 1) 14.2 and 16.9
template <int FMT, bool FUSED>
fp8q_status run_fp4(const void* t, const void* w, Fp4Args& p, cudaStream_t stream) {
  const int64_t sms = num_sms(), nw = FUSED ? p.I : p.N;
  auto rounds = [&](int64_t tiles) { return (tiles + sms - 1) / sms; };
  // token tiles: at most this many (an expert's last one may be ragged)
  const int64_t tt = p.offsets ? p.M / 128 + (p.M < p.E ? p.M : p.E) : (p.M + 127) / 128;
  const int64_t u128 = tt * ((nw + 127) / 128), u256 = tt * ((nw + 255) / 256);
  const int64_t per = p.offsets ? (p.M + p.E - 1) / p.E : p.M;      // rows of an expert, on average
  p.box = per > 64 ? 128 : p.M <= 16 ? 16 : 32;
  if (2 * u128 <= sms) return launch_fp4<FMT, 128, FUSED, false, true>(t, w, tt, p, stream);
  if constexpr (FUSED) {
    return launch_fp4<FMT, 128, true, false, false>(t, w, tt, p, stream);
  } else {
    if (p.offsets && per >= 768) {
      Fp4Args rest = p;
      p.share = kPairs;
      const fp8q_status st = launch_fp4<FMT, 256, false, true, false>(t, w, p.M / 129, p, stream);
      if (st != FP8Q_OK) return st;
      rest.share = kRest;
      rest.box = 32;
      return launch_fp4<FMT, 256, false, false, false>(t, w, p.M < p.E ? p.M : p.E, rest, stream);
    }
    const int64_t pairs = (p.M + 255) / 256 * ((nw + 255) / 256);
    if (!p.offsets && p.M > 128 && 2 * pairs >= sms)
      return launch_fp4<FMT, 256, false, true, false>(t, w, (p.M + 255) / 256, p, stream);
    if (2 * rounds(u256) > rounds(u128)) return launch_fp4<FMT, 128, false, false, false>(t, w, tt, p, stream);
    return launch_fp4<FMT, 256, false, false, false>(t, w, tt, p, stream);
  }
}

// Sizes, alignment and the argument block shared by the entry points.  Row
// coordinates and tile counts are 32 bits.
constexpr int64_t kMax32 = int64_t{1} << 31;

fp8q_status check_mm(const void* a_q, const void* b_q, const uint8_t* a_sf, const uint8_t* b_sf, int format,
                     const float* ga, const float* gb, int64_t E, int64_t M, int64_t N, int64_t K, Fp4Args* p) {
  if (format != FP8Q_FP4_NV && format != FP8Q_FP4_MX) return FP8Q_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || K <= 0 || N % 16 != 0 || K % 32 != 0 || E <= 0) return FP8Q_ERR_INVALID_ARG;
  if (E > kMaxExperts) return FP8Q_ERR_UNSUPPORTED;
  if (format == FP8Q_FP4_MX && (ga || gb)) return FP8Q_ERR_INVALID_ARG;
  if (M >= kMax32 || N >= kMax32 || K >= kMax32 || E * N >= kMax32 || (M / 128 + E) * ((N + 63) / 64) >= kMax32)
    return FP8Q_ERR_INVALID_ARG;
  if (M == 0) return FP8Q_OK;
  if (!a_q || !b_q || !a_sf || !b_sf) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_sf, 16) || !aligned(b_sf, 16) || !aligned(ga, 4) ||
      !aligned(gb, 4))
    return FP8Q_ERR_INVALID_ARG;
  p->M = M;
  p->N = N;
  p->K = K;
  p->sft = a_sf;
  p->sfw = b_sf;
  p->kb = static_cast<int>(fp4_kblocks(format, K));
  p->kstages = static_cast<int>((K + 255) / 256);
  p->wblocks = (N + 127) / 128;
  p->ga = ga;
  p->gb = gb;
  p->E = static_cast<int>(E);
  p->status = device_status_ptr();
  return FP8Q_OK;
}

fp8q_status check_y(void* y, int64_t ldy, int64_t M, int64_t N, Fp4Args* p) {
  if (ldy < N || ldy % 8 != 0 || (M > 0 && (!y || !aligned(y, 16)))) return FP8Q_ERR_INVALID_ARG;
  p->y = static_cast<uint16_t*>(y);
  p->ldy = ldy;
  return FP8Q_OK;
}

fp8q_status check_groups(const int* offsets, const int* sf_offsets, int64_t M, Fp4Args* p) {
  if (M > 0 && (!offsets || !sf_offsets || !aligned(offsets, 4) || !aligned(sf_offsets, 4)))
    return FP8Q_ERR_INVALID_ARG;
  p->offsets = offsets;
  p->sf_offsets = sf_offsets;
  return FP8Q_OK;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_scaled_mm_fp4(const void* a_q, const void* b_q, const uint8_t* a_sf, const uint8_t* b_sf,
                                          int format, const float* a_gscale, const float* b_gscale, int64_t M,
                                          int64_t N, int64_t K, void* y, int64_t ldy, void* stream) {
  Fp4Args p{};
  fp8q_status st = check_mm(a_q, b_q, a_sf, b_sf, format, a_gscale, b_gscale, 1, M, N, K, &p);
  if (st == FP8Q_OK) st = check_y(y, ldy, M, N, &p);
  if (st != FP8Q_OK || M == 0) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? run_fp4<kNv, false>(a_q, b_q, p, s) : run_fp4<kMx, false>(a_q, b_q, p, s);
}

extern "C" fp8q_status fp8q_grouped_mm_fp4(const void* a_q, const void* b_q, const uint8_t* a_sf, const uint8_t* b_sf,
                                           int format, const float* a_gscale, const float* b_gscale, const int* offsets,
                                           const int* sf_offsets, int64_t E, int64_t M, int64_t N, int64_t K, void* y,
                                           int64_t ldy, void* stream) {
  Fp4Args p{};
  fp8q_status st = check_mm(a_q, b_q, a_sf, b_sf, format, a_gscale, b_gscale, E, M, N, K, &p);
  if (st == FP8Q_OK) st = check_y(y, ldy, M, N, &p);
  if (st == FP8Q_OK) st = check_groups(offsets, sf_offsets, M, &p);
  if (st != FP8Q_OK || M == 0) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? run_fp4<kNv, false>(a_q, b_q, p, s) : run_fp4<kMx, false>(a_q, b_q, p, s);
}

extern "C" fp8q_status fp8q_grouped_mm_fp4_silu_quant(const void* a_q, const void* b_q, const uint8_t* a_sf,
                                                      const uint8_t* b_sf, int format, const float* a_gscale,
                                                      const float* b_gscale, const int* offsets, const int* sf_offsets,
                                                      int64_t E, int64_t M, int64_t I, int64_t K, const float* gscale,
                                                      void* q, uint8_t* sf, void* stream) {
  if (I <= 0 || I >= kMax32) return FP8Q_ERR_INVALID_ARG;
  Fp4Args p{};
  fp8q_status st = check_mm(a_q, b_q, a_sf, b_sf, format, a_gscale, b_gscale, E, M, 2 * I, K, &p);
  if (st == FP8Q_OK && I % 128 != 0) st = FP8Q_ERR_UNSUPPORTED;
  if (st == FP8Q_OK) st = check_groups(offsets, sf_offsets, M, &p);
  if (st != FP8Q_OK) return st;
  if (format == FP8Q_FP4_MX && gscale) return FP8Q_ERR_INVALID_ARG;
  if (M == 0) return FP8Q_OK;
  if (!q || !sf || !aligned(q, 16) || !aligned(sf, 16) || !aligned(gscale, 4)) return FP8Q_ERR_INVALID_ARG;
  p.I = I;
  p.hq = static_cast<uint8_t*>(q);
  p.hsf = sf;
  p.gh = gscale;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return format == FP8Q_FP4_NV ? run_fp4<kNv, true>(a_q, b_q, p, s) : run_fp4<kMx, true>(a_q, b_q, p, s);
}
