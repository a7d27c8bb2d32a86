// Attention over the rotated int8 cache for many rows: trees of drafted tokens and
// chunks, on the 5th-generation tensor cores. The mathematics, the line of work
// and the join are those of cache_attention.cu; a tile is 128 query rows by 128 keys.
//
// Here a key is read for 128 rows, so the softmax bounds it, as in the dense INT8
// attention: one exponential per row and key and five or six instructions beside it.
// (Times are of the device, for captured calls, unless they say otherwise.)
// One CTA per SM, two pipelines in it that take turns over the key tiles, so that
// one's softmax runs while the other's products do; each has its own sums (O in
// TMEM, reference and row sum in registers), joined at the end of a run:
//   warps 0-3, 4-7 : softmax of pipeline 0 and 1, a query row per thread: S from
//                    TMEM, logits, weights p s_v in fp16 into swizzled shared memory;
//   warps 8-11     : the tile's values, widened exactly from int8 to fp16 into the
//                    (MN-major) operand of P V, and its scales; the loads run a
//                    tile and two tiles ahead;
//   warp 12        : key codes by TMA (boxes of 16 keys: pages are no smaller);
//   warp 13        : issues S = Q K^T (kind::i8, 128 x 128 x 128) and O += P V
//                    (kind::f16, fp16 operands).
// A tile is one pass over its logits at the row's reference, 16 keys at a time. The
// roles of a CTA run different code at once, and what they share is the instruction
// cache: with a row's 128 logits in registers, and their maximum taken first, a tile
// took 3.8 us; rolled over 64 keys the trees of 8 sequences took 61 us, over 32 57.6, over
// 16 54.6, with the values' loop rolled too 54.3. Splitting a tile into halves with barriers
// of their own, so that one half's products run during the other's softmax, cost more in
// code than it hid (58.7).
// The reference is chosen so that the weights, not the exponentials, fit fp16: the
// largest weight so far lies between 1 and 2^15, whatever the range of the value
// scales. A row whose weights have grown takes it up at the next tile (that alone:
// 67 to 60 us for a tree of 64 drafts behind 32768 keys); only where a weight passes
// 2^15 within one tile, or a row's first ones are far below their bound, is the tile taken
// again, at a reference from the logit and scale of each key.
// Rounding a weight to fp16 is far below bf16's own rounding of the output. For an fp16 output it
// is as large (2.9e-4 of a row against 2.1e-4 without it), so there a second product adds what the first rounding
// left, as in the kernel for few rows. Both operands of a whole tile do not fit beside the rest of the shared
// memory: the tile is taken in two steps of 64 keys, which costs the tree of 64 drafts behind 32768 keys 60 us
// for 49.
// A run costs about as much as three tiles beside its tiles. Its first two tiles' keys
// are fetched before its queries are in place, their pages looked up by eight lanes at
// once, and the parts it leaves for the join lie four channels of all rows after one
// another, so that both sides move whole lines: 54.3 to 43.9 us for the trees of 8
// sequences (42.5 since the warps keep the registers they are launched with: handing
// some of the others' to the softmax warps gained nothing. 14 warps are allocated as 16, so
// that a thread has 128 registers and spills 200 to 220 bytes, most of them once a run or tile).
// What holds every wait, reference and sum right, wherever they lie, took it from there to 45.4.
// What bounds a tile now (2 us per SM): the latencies of a pass, 1024 cycles of
// which are the exponentials, and between passes the turn of the products, which need the
// logits read before the next are made.
// Every wait is bounded. Once one has run out, the CTA's roles leave the walk together at
// the end of the run, with the barriers' phases still agreed, and the softmax warps go on alone: the rows
// of that run and of the piece's later ones become NaN, also where the join sums them.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "cache_attention.cuh"
#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"
#include "ptx_sm100.cuh"

namespace convrot {

namespace {

constexpr int CW_KT = 128;           // keys of a tile
constexpr int CW_THREADS = 448;
constexpr int CW_HALF = 128 * 128;   // 128 rows of 128 bytes
// a run costs about as much as three tiles beside its tiles
using CwGrain = CaGrain<CA_WIDE_ROWS, CW_KT, 3, 2>;
constexpr uint32_t CW_IDESC_S = idesc_i8(128, CW_KT);
// fp16 operands, float32 sums, 128 x 128, B MN-major
constexpr uint32_t CW_IDESC_O = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr float CW_MOST = 32768.0f;  // weights stay below 2^15
constexpr float CW_GROWN = 16.0f;    // past it a row's reference goes up at the next tile
constexpr float CW_SPAN = 100.0f;    // exponentials below 2^100
constexpr float CW_FAR = 0x1p24f;    // logits from here on differ by whole numbers

struct CwSmem {
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + CW_HALF;            // two pipelines
  static constexpr int kOffP = kOffK + 2 * CW_HALF;
  static constexpr int kOffV = kOffP + 2 * 2 * CW_HALF;
  static constexpr int kOffScale = kOffV + 2 * 2 * CW_HALF;  // [pipeline][buffer] 128 key, 128 value scales
  static constexpr int kOffTile = kOffScale + 2 * 2 * 256 * 4;  // [pipeline][buffer] 4 words of keys there, 4 largest value scales
  static constexpr int kOffRow = kOffTile + 2 * 2 * 8 * 4;   // query factors
  static constexpr int kOffStat = kOffRow + 128 * 4;         // [pipeline][row] maximum, sum
  static constexpr int kOffScan = kOffStat + 2 * 128 * 8;
  // per pipeline: keys there, keys read, S there, S read, values there, scales there (of each buffer), weights there and
  // P V done (of each step); then drain
  static constexpr int kOffBar = kOffScan + 18 * 8;
  static constexpr int kBarriers = 23;
  static constexpr int kOffMisc = kOffBar + kBarriers * 8 + 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

enum CwBar { kKFull, kKEmpty, kSFull, kSEmpty, kVFull, kSc0, kSc1, kPFull, kPFull1, kODone, kODone1, kBars };
static_assert(2 * kBars + 1 == CwSmem::kBarriers, "room for the barriers");

// A barrier of whole warps: what stands before it may have been single lanes' work.
__device__ __forceinline__ void cw_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same barrier, and whether any of its threads brought a true.
__device__ __forceinline__ bool cw_vote(int id, int threads, bool mine) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(mine ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return any != 0;
}

// A word of the keys below `n` among keys 32 w .. 32 w + 31 of a tile.
__device__ __forceinline__ uint32_t below(int n, int w) {
  const int m = n - 32 * w;
  return m <= 0 ? 0u : m >= 32 ? 0xFFFFFFFFu : (1u << m) - 1u;
}

// Word w of 64 bits placed at bit `at` (which may be negative) of a tile's keys.
__device__ __forceinline__ uint32_t placed(unsigned long long bits, int at, int w) {
  const int shift = 32 * w - at;  // the word's first key is this bit
  if (shift >= 64 || shift <= -32) return 0u;
  return static_cast<uint32_t>(shift >= 0 ? bits >> shift : bits << -shift);
}

// Two sums of 128 products of codes (|acc| < 2^22) as floats times the keys' scales, without a conversion
// instruction: the integer added to the bits of 1.5 * 2^23 is exact, and so is subtracting 1.5 * 2^23.
__device__ __forceinline__ float2 cw_logits(uint32_t a, uint32_t b, float2 scale) {
  const float2 x = make_float2(__uint_as_float(a + 0x4B400000u), __uint_as_float(b + 0x4B400000u));
  return __fmul2_rn(__fadd2_rn(x, make_float2(-12582912.0f, -12582912.0f)), scale);
}

// Exponent of a positive float: 2^e <= x < 2^(e + 1).
__device__ __forceinline__ float exponent_of(float x) {
  return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127);
}

// The row's functions below work on one step of a tile: CHUNKS times 16 keys, from 16 w0 on.

// The largest logit of a row among the keys it sees, without the row's factor.
template <int CHUNKS>
__device__ __forceinline__ float cw_top(uint32_t tS, const uint32_t (&vis)[4], const float* sk, int w0) {
  float top = -INFINITY;
#pragma unroll 1
  for (int w = w0 >> 1; w < (w0 + CHUNKS) >> 1; ++w) {
    uint32_t a[32];
    tmem_ld_32x32b_x32(tS + w * 32, a);
    const uint32_t on = w == 0 ? vis[0] : w == 1 ? vis[1] : w == 2 ? vis[2] : vis[3];
    tmem_ld_wait_regs(a);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float2 u = cw_logits(a[k], a[k + 1], *reinterpret_cast<const float2*>(sk + w * 32 + k));
      top = fwht::fmax3f(top, on >> k & 1u ? u.x : -INFINITY, on >> (k + 1) & 1u ? u.y : -INFINITY);
    }
  }
  return top;
}

// The reference at which a row's largest weight among the keys it sees lies near 2, unless exponentials would pass
// 2^CW_SPAN: from the logit and the scale of each key. Past CW_FAR, where a logit has no bits left for the scale's
// exponent beside it, the largest logit, and apart from it in `lift` what the reference should lie above it.
template <int CHUNKS>
__device__ __forceinline__ float cw_exact(uint32_t tS, float c, const uint32_t (&vis)[4], const float* sk, int w0,
                                          float* lift) {
  float top = -INFINITY, heavy = -INFINITY;
#pragma unroll 1
  for (int w = w0; w < w0 + CHUNKS; ++w) {
    uint32_t a[16];
    tmem_ld_32x32b_x16(tS + w * 16, a);
    const uint32_t on = (w < 4 ? (w < 2 ? vis[0] : vis[1]) : (w < 6 ? vis[2] : vis[3])) >> (16 * (w & 1));
    tmem_ld_wait_regs16(a);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float2 u = cw_logits(a[k], a[k + 1], *reinterpret_cast<const float2*>(sk + w * 16 + k));
      const float2 v = *reinterpret_cast<const float2*>(sk + 128 + w * 16 + k);
      const float x = on >> k & 1u ? c * u.x : -INFINITY, y = on >> (k + 1) & 1u ? c * u.y : -INFINITY;
      top = fwht::fmax3f(top, x, y);
      // the exponent's bits as the last ones of 2^23: the sum is rounded to a whole number
      heavy = fwht::fmax3f(heavy, x + __uint_as_float(0x4B000000u | (__float_as_uint(v.x) >> 23 & 255u)),
                           y + __uint_as_float(0x4B000000u | (__float_as_uint(v.y) >> 23 & 255u)));
    }
  }
  const float at = fmaxf(heavy - (8388608.0f + 127.0f + 1.0f), top - CW_SPAN);
  const bool far = fabsf(top) > CW_FAR && top > -INFINITY;
  *lift = 0.0f;
  if (__any_sync(0xFFFFFFFFu, far)) {
    heavy = -INFINITY;
#pragma unroll 1
    for (int w = w0; w < w0 + CHUNKS; ++w) {
      uint32_t a[16];
      tmem_ld_32x32b_x16(tS + w * 16, a);
      const uint32_t on = (w < 4 ? (w < 2 ? vis[0] : vis[1]) : (w < 6 ? vis[2] : vis[3])) >> (16 * (w & 1));
      tmem_ld_wait_regs16(a);
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float2 u = cw_logits(a[k], a[k + 1], *reinterpret_cast<const float2*>(sk + w * 16 + k));
        const float2 v = *reinterpret_cast<const float2*>(sk + 128 + w * 16 + k);
        const float x = __fadd_rn(__fmul_rn(c, u.x), -top) + exponent_of(v.x);
        const float y = __fadd_rn(__fmul_rn(c, u.y), -top) + exponent_of(v.y);
        heavy = fwht::fmax3f(heavy, on >> k & 1u ? x : -INFINITY, on >> (k + 1) & 1u ? y : -INFINITY);
      }
    }
    if (far) *lift = fmaxf(heavy - 1.0f, -CW_SPAN);
  }
  return far ? top : at;
}

// One pass over a tile's logits: the weights of the row in fp16 into its line of the operand, the sum of the
// exponentials, and the largest weight. A logit's product is not rounded before the reference is taken off, which was;
// past CW_FAR that difference could leave float32's exponents, and FAR rounds both alike (everywhere it took 3 % longer),
// and takes off the lift, which is 0 for other rows.
// With REST the operand's second half holds what rounding the weights of the first left.
template <bool MASKED, bool FAR, bool REST>
__device__ __forceinline__ void cw_pass(uint32_t tS, float c, float ref, float lift, const uint32_t (&vis)[4],
                                        const float* sk, uint8_t* line, int sw, int w0, float* sum, float* most) {
  const float* sv = sk + 128;
  const float2 c2 = make_float2(c, c), nref = make_float2(-ref, -ref);
  float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  float big[2] = {0.0f, 0.0f};
#pragma unroll 1
  for (int w = w0; w < w0 + (REST ? 4 : 8); ++w) {
    uint32_t a[16];
    tmem_ld_32x32b_x16(tS + w * 16, a);
    float4 fks[4], fvs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fks[i] = *reinterpret_cast<const float4*>(sk + w * 16 + 4 * i);
      fvs[i] = *reinterpret_cast<const float4*>(sv + w * 16 + 4 * i);
    }
    tmem_ld_wait_regs16(a);
    const uint32_t on = (w < 4 ? (w < 2 ? vis[0] : vis[1]) : (w < 6 ? vis[2] : vis[3])) >> (16 * (w & 1));
    uint8_t* to = line + (!REST && w >= 4 ? CW_HALF : 0);
    const int c0 = 2 * (w & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t out[4], rest[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 fk = fks[2 * i + q], fv = fvs[2 * i + q];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = i * 8 + 4 * q + 2 * e;
          const float2 u = cw_logits(a[k], a[k + 1], e == 0 ? make_float2(fk.x, fk.y) : make_float2(fk.z, fk.w));
          const float2 t = FAR ? make_float2(__fadd_rn(__fmul_rn(c, u.x), -ref) - lift,
                                             __fadd_rn(__fmul_rn(c, u.y), -ref) - lift)
                               : __ffma2_rn(c2, u, nref);
          float2 pr = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          float2 x = __fmul2_rn(pr, e == 0 ? make_float2(fv.x, fv.y) : make_float2(fv.z, fv.w));
          if (MASKED) {
            const bool y = on >> k & 1u, z = on >> (k + 1) & 1u;
            pr = make_float2(y ? pr.x : 0.0f, z ? pr.y : 0.0f);
            x = make_float2(y ? x.x : 0.0f, z ? x.y : 0.0f);
          }
          part[e] = __fadd2_rn(part[e], pr);
          big[e] = fwht::fmax3f(big[e], x.x, x.y);
          const __half2 hx = __floats2half2_rn(x.x, x.y);
          out[2 * q + e] = *reinterpret_cast<const uint32_t*>(&hx);
          if (REST) {
            const float2 f = __half22float2(hx);
            const __half2 hr = __floats2half2_rn(x.x - f.x, x.y - f.y);
            rest[2 * q + e] = *reinterpret_cast<const uint32_t*>(&hr);
          }
        }
      }
      *reinterpret_cast<uint4*>(to + (((c0 + i) ^ sw) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
      if (REST)
        *reinterpret_cast<uint4*>(to + CW_HALF + (((c0 + i) ^ sw) << 4)) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
  }
  const float2 all = __fadd2_rn(part[0], part[1]);
  *sum = all.x + all.y;
  *most = fmaxf(big[0], big[1]);
}

// A row's sums of values in TMEM by a factor.
__device__ __forceinline__ void cw_scale(uint32_t tO, float by) {
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(tO + ch * 32, o);
    tmem_ld_wait_regs(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
    tmem_st_32x32b_x32(tO + ch * 32, o);
  }
  tmem_st_wait();
}

template <bool F16>
__global__ void __launch_bounds__(CW_THREADS, 1)
    cache_attention_wide_kernel(const __grid_constant__ CUtensorMap tmK, const CaParams p) {
  using L = CwSmem;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, not through an integer, so that the compiler still knows it is shared memory
  uint8_t* smem = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* drain = bars + 2 * kBars;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kOffMisc);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int pipe, int which) { return bars + pipe * kBars + which; };

  // For an fp16 output, which keeps as many bits as a weight, a tile is taken in two steps of 64 keys, whose operand
  // holds beside the weights what rounding them left.
  constexpr int STEPS = F16 ? 2 : 1, CHUNKS = 8 / STEPS;
  constexpr int kOLast = kODone + STEPS - 1;

  griddep_launch_dependents();
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    for (int pipe = 0; pipe < 2; ++pipe) {
      mbar_init(bar(pipe, kKFull), 1);
      mbar_init(bar(pipe, kKEmpty), 1);
      mbar_init(bar(pipe, kSFull), 1);
      mbar_init(bar(pipe, kSEmpty), 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(pipe, kPFull + h), 4);
        mbar_init(bar(pipe, kODone + h), 1);
      }
      mbar_init(bar(pipe, kVFull), 4);
      mbar_init(bar(pipe, kSc0), 4);
      mbar_init(bar(pipe, kSc1), 4);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_ptr, 512);
    tmem_relinquish();
  }
  int bad = 0;
  CaWalk<CwGrain> walk{};
  const int64_t per = ca_piece<CwGrain, CW_THREADS>(p, reinterpret_cast<int64_t*>(smem + L::kOffScan), &walk, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;  // S of the two pipelines, then O

  // A wait of the role; false once one has run out anywhere in the CTA.
  auto wait = [&](uint64_t* b, int use) {
    const uint32_t parity = static_cast<uint32_t>(use & 1);
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_suspend(b, parity, p.wait_step)) {
      if (*abort || global_timer_ns() - t0 > p.wait_ns) {
        *abort = 1;
        bad |= CA_LATE;
        return false;
      }
    }
    return true;
  };
  // Tiles that a pipeline has taken in earlier runs: the parity of its barriers. Every role counts alike, and
  // meets the others twice a run (barrier 0): the queries are in place; the sums have been read, and whether a
  // wait has run out is known to all.
  int used[2] = {0, 0};
  CaRun r;
  CaCut cut{};

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int pipe = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + pipe * 128, tO = tmem + lanes + 256 + pipe * 128;
    uint8_t* line = smem + L::kOffP + pipe * 2 * CW_HALF + row * 128;
    const int sw = row & 7;
    float* row_c = reinterpret_cast<float*>(smem + L::kOffRow);
    float2* stat = reinterpret_cast<float2*>(smem + L::kOffStat);
    // A run up to its sums, in stat and TMEM; false once a wait has run out in the CTA.
    auto sums = [&]() {
      const int keys = walk.s.keys, context = keys - walk.s.news;
      if (p.tree != nullptr && walk.s.news > 64) bad |= CA_BAD;
      // the tile's queries, rotated and quantised: four lanes a row, 16 rows a warp
      {
        const int l4 = lane & 3;
        uint4 w[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = warp * 16 + k * 8 + (lane >> 2);
          const int of = r.row0 + at, i = of / p.G;
          const uint16_t* src = p.q + (walk.s.first + i) * p.qt + (r.head * p.G + (of - i * p.G)) * p.qh + 8 * l4;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[k][j] = at < r.rows ? __ldg(reinterpret_cast<const uint4*>(src + 32 * j)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = warp * 16 + k * 8 + (lane >> 2);
          float2 v[16];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {w[k][j].x, w[k][j].y, w[k][j].z, w[k][j].w};
            const uint32_t b[4] = {w[k][2 + j].x, w[k][2 + j].y, w[k][2 + j].z, w[k][2 + j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              fwht::fwht_first_pair<F16>(a[e], fwht::widen_pair<F16>(b[e]), v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
          }
          fwht::fwht128_quad(v, l4);
          float amax = fabsf(v[0].x);  // NaN where all are
#pragma unroll
          for (int i = 0; i < 16; ++i) amax = fwht::fmax3f(amax, fabsf(v[i].x), fabsf(v[i].y));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
          const fwht::CodeFactor f = fwht::code_factor(amax);
          const float2 ci = make_float2(f.ci, f.ci), pre = make_float2(f.pre, f.pre);
          const float2 magic = make_float2(fwht::kRoundMagic, fwht::kRoundMagic);
          uint8_t* line_q = smem + L::kOffQ + at * 128 + (l4 & 1) * 8;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __ffma2_rn(__fmul2_rn(v[8 * j + e], pre), ci, magic);
            // channels 32 j + 8 l4 .. + 7 and 64 more: half of a 16-byte chunk each
            *reinterpret_cast<uint2*>(line_q + (((2 * j + (l4 >> 1)) ^ (at & 7)) << 4)) =
                make_uint2(fwht::pack4(x[0].x, x[1].x, x[2].x, x[3].x), fwht::pack4(x[4].x, x[5].x, x[6].x, x[7].x));
            *reinterpret_cast<uint2*>(line_q + (((4 + 2 * j + (l4 >> 1)) ^ (at & 7)) << 4)) =
                make_uint2(fwht::pack4(x[0].y, x[1].y, x[2].y, x[3].y), fwht::pack4(x[4].y, x[5].y, x[6].y, x[7].y));
          }
          if (l4 == 0) row_c[at] = ca_query_factor(p, amax);
        }
      }
      fence_proxy_async_smem();
      cw_sync(0, CW_THREADS);

      const float c = row_c[row];  // >= 0 or NaN
      int lim = 0;                 // keys below it are seen, and with a tree the drafted keys whose bit is set
      unsigned long long bits = 0;
      {
        const int i = row < r.rows ? (r.row0 + row) / p.G : 0;
        lim = p.tree != nullptr ? context : context + i + 1;
        if (p.tree != nullptr && row < r.rows) bits = __ldg(p.tree + walk.s.first + i);
      }
      const int clear = p.tree != nullptr ? context : context + 1;  // keys below it are seen by every row
      float ref = CA_NONE, l = 0.0f, largest = 0.0f;
      bool weighed = false;  // the row has had a weight
      // A row of the warp has a reference past CW_FAR, which is then the sum of ref and lift (0 in other rows). That
      // costs bf16 trees of 8 sequences 45.4 us of device time for 43.7, by registers.
      bool far = false;
      float lift = 0.0f;
      bool ok = true;
      int use = used[pipe];
      for (int t = r.t0 + pipe; t < r.t1; t += 2, ++use) {
        const int key0 = t * CW_KT;
        const int buffer = pipe * 2 + (use & 1);
        const float* sk = reinterpret_cast<const float*>(smem + L::kOffScale) + buffer * 256;
        const uint32_t* there = reinterpret_cast<const uint32_t*>(smem + L::kOffTile) + buffer * 8;
        const float* most = reinterpret_cast<const float*>(there + 4);
        ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kSc0 + (use & 1)), use >> 1) && wait(bar(pipe, kSFull), use));
        if (!ok) break;
        uint32_t vis[4] = {there[0], there[1], there[2], there[3]};
        const bool masked = key0 + CW_KT > clear || (vis[0] & vis[1] & vis[2] & vis[3]) != 0xFFFFFFFFu;
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w) vis[w] &= below(lim - key0, w) | placed(bits, context - key0, w);
        }
#pragma unroll 1
        for (int step = 0; step < STEPS; ++step) {
          const int w0 = step * CHUNKS;
          // the pipeline's last P V has finished: O is stable and the operand's memory free
          if (step > 0 || use > 0) {
            ok = __all_sync(0xFFFFFFFFu, step > 0 ? wait(bar(pipe, kODone), use) : wait(bar(pipe, kOLast), use - 1));
            if (!ok) break;
          }
          tc_fence_after();
          const float high = STEPS == 1 ? fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]))
                                        : fmaxf(most[2 * step], most[2 * step + 1]);
          const uint32_t any = STEPS == 1 ? vis[0] | vis[1] | vis[2] | vis[3] : step == 0 ? vis[0] | vis[1] : vis[2] | vis[3];
          const bool first = !weighed && any != 0;
          // the sum so far may be of keys without a value, and must stay in range where the reference comes down
          const float least = !(l > 0.0f) ? CA_NONE : fabsf(ref) > CW_FAR ? ref : ref + exponent_of(l) - CW_SPAN;
          float now = ref, now_lift = lift, sum, big;
          // A row whose weights have grown takes its reference up before they can pass fp16's range: one
          // rescaling of O instead of a second pass.
          if (largest > CW_GROWN) (far && fabsf(ref) > CW_FAR ? now_lift : now) += exponent_of(largest);
          if (__any_sync(0xFFFFFFFFu, first)) {
            // at this every weight of the tile is below 2^8, the largest usually little below
            const float tm = c * cw_top<CHUNKS>(tS, vis, sk, w0);
            if (first) {
              now = fabsf(tm) > CW_FAR ? fmaxf(tm, least)
                                       : fmaxf(high > 0.0f ? tm + exponent_of(high) - 7.0f : tm, fmaxf(tm - CW_SPAN, least));
              if (!(fabsf(now) > CW_FAR)) now_lift = 0.0f;
            }
            far = __any_sync(0xFFFFFFFFu, fabsf(now) > CW_FAR && now != CA_NONE);
          }
#pragma unroll 1
          for (int attempt = 0;; ++attempt) {
            __syncwarp();  // a pass is the whole warp's; what led here differs by row
            if (far) cw_pass<true, true, F16>(tS, c, now, now_lift, vis, sk, line, sw, w0, &sum, &big);
            else if (masked) cw_pass<true, false, F16>(tS, c, now, 0.0f, vis, sk, line, sw, w0, &sum, &big);
            else cw_pass<false, false, F16>(tS, c, now, 0.0f, vis, sk, line, sw, w0, &sum, &big);
            const bool lost = !(big <= CW_MOST) || !(sum <= 0x1p110f) || (first && high > 0.0f && big < 1.0f);
            if (attempt == 1 || !__any_sync(0xFFFFFFFFu, lost)) break;
            float up;
            const float at = cw_exact<CHUNKS>(tS, c, vis, sk, w0, &up);
            if (lost) {
              now = fmaxf(at, least);
              now_lift = 0.0f;
              if (fabsf(now) > CW_FAR && now != CA_NONE)  // the sum so far must stay in range here as well
                now_lift = fmaxf(up + (at - now), l > 0.0f ? ref - now + lift + exponent_of(l) - CW_SPAN : -CW_SPAN);
            }
            far = __any_sync(0xFFFFFFFFu, fabsf(now) > CW_FAR && now != CA_NONE);
          }
          weighed |= big > 0.0f;
          // in two factors for the sum: one of up to 2^110 may count where a single factor is lost below 2^-126
          const float half = ex2_approx(0.5f * (ref - now + (lift - now_lift))), scale = half * half;
          largest = fmaxf(largest * scale, big);
          const float alpha = ref == CA_NONE ? (now == ref ? 1.0f : 0.0f) : scale;
          ref = now;
          lift = now_lift;
          l = l * half * half + sum;
          // the logits have been read, the operand is in place, and O has the new reference
          if ((step > 0 || t >= r.t0 + 2) && __any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
            cw_scale(tO, alpha);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (step == STEPS - 1) mbar_arrive(bar(pipe, kSEmpty));
            mbar_arrive(bar(pipe, kPFull + step));
          }
        }
        if (!ok) break;
      }
      const int mine = r.t1 - r.t0 > pipe ? (r.t1 - r.t0 - pipe + 1) / 2 : 0;
      if (ok && mine > 0) ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kOLast), used[pipe] + mine - 1));
      if (ok && far) {
        // the join knows one number for a reference: back to the logit's
        tc_fence_after();
        const float half = ex2_approx(0.5f * lift);
        cw_scale(tO, half * half);
        l = l * half * half;
      }
      stat[pipe * 128 + row] = make_float2(ref, l);
      tc_fence_before();
      const bool lost = cw_vote(1, 256, !ok);
      tc_fence_after();
      return !lost;
    };
    bool dead = false;
    while (walk.next(p, &r, bad)) {
      if (walk.s.keys == 0) {  // nothing to see: zeros
        for (int i = tid; i < r.rows * (CA_D / 8); i += 256) {
          const int of = r.row0 + i / (CA_D / 8), token = of / p.G;
          *reinterpret_cast<uint4*>(p.o + (walk.s.first + token) * p.ot + (r.head * p.G + (of - token * p.G)) * p.oh +
                                    8 * (i % (CA_D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const bool there = !dead && sums();
      // ---- the pipelines joined; channels 0 .. 63 here, 64 .. 127 in the other pipeline's warps
      const bool second = r.t1 - r.t0 > 1;
      const float2 s0 = stat[row], s1 = second ? stat[128 + row] : make_float2(CA_NONE, 0.0f);
      const float top = fmaxf(s0.x, s1.x);
      const float h0 = ex2_approx(0.5f * (s0.x - top)), h1 = ex2_approx(0.5f * (s1.x - top));  // halves, as above
      const float f0 = h0 * h0, f1 = h1 * h1;
      const float total = s0.y * h0 * h0 + s1.y * h1 * h1;
      const bool whole = r.t0 == 0 && r.t1 == walk.s.tiles;
      const uint32_t tO0 = tmem + lanes + 256, tO1 = tO0 + 128;
      if (!there) {
        if (pipe == 0 && row < r.rows) {
          if (whole) {
            const int of = r.row0 + row, i = of / p.G;
            uint16_t* dst = p.o + (walk.s.first + i) * p.ot + (r.head * p.G + (of - i * p.G)) * p.oh;
            for (int k = 0; k < CA_D / 8; ++k)  // NaN in either type
              *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
          } else {
            // a sum that is no number makes the row none, whatever its channels hold
            p.part_ml[(2 * static_cast<int64_t>(blockIdx.x) + (r.t0 == 0 ? 1 : 0)) * CA_WIDE_ROWS + row] =
                make_float2(0.0f, __uint_as_float(0x7FFFFFFFu));
          }
        }
      } else if (!whole) {
        // this half's channels, unnormalised; rolled, for the instruction cache
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (r.t0 == 0 ? 1 : 0);
        // four channels of all rows after one another, so that a warp's stores are contiguous
        float4* dst = reinterpret_cast<float4*>(p.part) + (slot * (CA_D / 4) + 16 * pipe) * CA_WIDE_ROWS + row;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch, dst += 4 * CA_WIDE_ROWS) {
          uint32_t a[16], b[16];
          tmem_ld_32x32b_x16(tO0 + 64 * pipe + ch * 16, a);
          if (second) tmem_ld_32x32b_x16(tO1 + 64 * pipe + ch * 16, b);
          tmem_ld_wait_regs16(a);
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(a[i]) * f0;
          if (second) {
            tmem_ld_wait_regs16(b);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(__uint_as_float(b[i]), f1, v[i]);
          }
          if (row < r.rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k * CA_WIDE_ROWS] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
          __syncwarp();
        }
        if (pipe == 0 && row < r.rows) p.part_ml[slot * CA_WIDE_ROWS + row] = make_float2(top, total);
      } else {
        // the last butterfly stage, between channels 64 apart, comes first
        float v[64];
        const float sign = pipe == 0 ? 1.0f : -1.0f;
        const float g0 = sign * f0, g1 = sign * f1;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t a[16], b[16];
          tmem_ld_32x32b_x16(tO0 + ch * 16, a);
          tmem_ld_32x32b_x16(tO0 + 64 + ch * 16, b);
          tmem_ld_wait_regs16(a);
          tmem_ld_wait_regs16(b);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[ch * 16 + i] = fmaf(__uint_as_float(b[i]), g0, __uint_as_float(a[i]) * f0);
          if (second) {
            tmem_ld_32x32b_x16(tO1 + ch * 16, a);
            tmem_ld_32x32b_x16(tO1 + 64 + ch * 16, b);
            tmem_ld_wait_regs16(a);
            tmem_ld_wait_regs16(b);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[ch * 16 + i] = fmaf(__uint_as_float(b[i]), g1, fmaf(__uint_as_float(a[i]), f1, v[ch * 16 + i]));
          }
        }
        const float norm = total == 0.0f ? 0.0f : fwht::kInvSqrt128 / total;
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = total == 0.0f ? 0.0f : v[i] * norm;
        fwht::reg_stage<64, 1>(v);
        fwht::reg_stage<64, 2>(v);
        fwht::reg_stage<64, 4>(v);
        fwht::reg_stage<64, 8>(v);
        fwht::reg_stage<64, 16>(v);
        fwht::reg_stage<64, 32>(v);
        if (row < r.rows) {
          const int of = r.row0 + row, i = of / p.G;
          uint16_t* dst = p.o + (walk.s.first + i) * p.ot + (r.head * p.G + (of - i * p.G)) * p.oh + 64 * pipe;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(
                fwht::narrow_pair<F16>(v[8 * k], v[8 * k + 1]), fwht::narrow_pair<F16>(v[8 * k + 2], v[8 * k + 3]),
                fwht::narrow_pair<F16>(v[8 * k + 4], v[8 * k + 5]), fwht::narrow_pair<F16>(v[8 * k + 6], v[8 * k + 7]));
        }
      }
      if (r.t0 == 0 && !whole) {
        // the piece ends inside an item that begins in it: it describes the item to the join
        cut.pieces = static_cast<int>((walk.end + r.left - 1) / per) - static_cast<int>(blockIdx.x) + 1;
        cut.rows = r.rows;
        cut.row0 = r.row0;
        cut.head = r.head;
        cut.token0 = walk.s.first;
      }
      if (dead) continue;
      used[0] += (r.t1 - r.t0 + 1) / 2;
      used[1] += (r.t1 - r.t0) / 2;
      tc_fence_before();
      dead = cw_vote(0, CW_THREADS, !there);
    }
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  } else if (warp < 12) {
    // ----------------------------------------------------------------- values
    const int me = tid - 256;  // the thread's key of a tile, for the scales
    const int w4 = warp - 8;
    while (walk.next(p, &r, bad)) {
      if (walk.s.keys == 0) continue;
      const int keys = walk.s.keys;
      const int32_t* table = p.pages + walk.b * p.table_stride;
      auto cell_of = [&](int key) {  // the cell of a key, or -1
        if (key >= keys) return -1;
        const int page = __ldg(table + (key >> p.page_shift));
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
          bad |= CA_BAD;  // its keys are not seen
          return -1;
        }
        return ((page * p.Hkv + r.head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
      };
      // Loads run ahead: codes one tile, scales two. Eight lanes a key, 16 codes each: keys w4 * 32 + 4 i + lane / 8.
      auto load_codes = [&](int cell_mine, uint4 (&code)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int cell = __shfl_sync(0xFFFFFFFFu, cell_mine, 4 * i + (lane >> 3));
          code[i] = cell >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.v_codes + static_cast<int64_t>(cell) * CA_D) +
                                      (lane & 7))
                              : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      auto load_scale = [&](const float* from, int cell) { return cell >= 0 ? __ldg(from + cell) : 0.0f; };
      auto give_scales = [&](int n, int cell, float mk, float mv) {  // tile n of the run
        // the buffer was last used two tiles of this pipeline ago, whose P V has been waited for
        const int pipe = n & 1, use = used[pipe] + (n >> 1), buffer = pipe * 2 + (use & 1);
        float* sk = reinterpret_cast<float*>(smem + L::kOffScale) + buffer * 256;
        uint32_t* there = reinterpret_cast<uint32_t*>(smem + L::kOffTile) + buffer * 8;
        sk[me] = mk;
        sk[128 + me] = mv;
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, cell >= 0);
        float most = fabsf(mv);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
        if (lane == 0) {
          there[w4] = on;
          reinterpret_cast<float*>(there + 4)[w4] = most;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(pipe, kSc0 + (use & 1)));
      };
      const int tiles = r.t1 - r.t0;
      // Tile n: the codes of the next into `other`, its scales, then this one's values; false once a wait has run out.
      int cell1 = -1, cell2 = -1;  // of this thread's key in the next tile and the one after
      float mk = 0.0f, mv = 0.0f;  // the next tile's scales
      auto tile = [&](int n, const uint4 (&code)[8], uint4 (&other)[8]) {
        const int pipe = n & 1, use = used[pipe] + (n >> 1);
        if (n + 1 < tiles) {
          load_codes(cell1, other);
          give_scales(n + 1, cell1, mk, mv);
          cell2 = n + 2 < tiles ? cell_of((r.t0 + n + 2) * CW_KT + me) : -1;
        }
        if (use > 0 && !__all_sync(0xFFFFFFFFu, wait(bar(pipe, kOLast), use - 1))) return false;
        uint8_t* to = smem + L::kOffV + pipe * 2 * CW_HALF + ((lane >> 2) & 1) * CW_HALF;  // channels from 64 on: second half
        const __half2 offset = __floats2half2_rn(1152.0f, 1152.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = w4 * 32 + 4 * i + (lane >> 3);
          const uint32_t word[4] = {code[i].x ^ 0x80808080u, code[i].y ^ 0x80808080u, code[i].z ^ 0x80808080u,
                                    code[i].w ^ 0x80808080u};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // fp16 of a code: the byte plus 128 in the low bits of 1024, minus 1152, exactly
            const uint32_t x = __byte_perm(word[e >> 1], 0x64646464u, e & 1 ? 0x4342 : 0x4140);
            const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&x), offset);
            h[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
          const int chunk = 2 * (lane & 3);
          *reinterpret_cast<uint4*>(to + key * 128 + ((chunk ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + key * 128 + (((chunk + 1) ^ (key & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(pipe, kVFull));
        cell1 = cell2;
        mk = load_scale(p.k_scale, cell1);
        mv = load_scale(p.v_scale, cell1);
        return true;
      };
      uint4 code_a[8], code_b[8];
      {
        const int cell0 = cell_of(r.t0 * CW_KT + me);
        cell1 = tiles > 1 ? cell_of((r.t0 + 1) * CW_KT + me) : -1;
        const float k0 = load_scale(p.k_scale, cell0), v0 = load_scale(p.v_scale, cell0);
        load_codes(cell0, code_a);
        mk = load_scale(p.k_scale, cell1);
        mv = load_scale(p.v_scale, cell1);
        give_scales(0, cell0, k0, v0);
      }
      cw_sync(0, CW_THREADS);
#pragma unroll 1
      for (int n = 0; n < tiles; ++n) {
        if (!tile(n, code_a, code_b)) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) code_a[i] = code_b[i];
      }
      used[0] += (r.t1 - r.t0 + 1) / 2;
      used[1] += (r.t1 - r.t0) / 2;
      if (cw_vote(0, CW_THREADS, (bad & 4) != 0)) break;  // a timeout is 5
    }
  } else {
    if (warp == 12) {
      // ------------------------------------------------------------------ keys
      int issued[2] = {0, 0};
      while (walk.next(p, &r, bad)) {
        if (walk.s.keys == 0) continue;
        const int32_t* table = p.pages + walk.b * p.table_stride;
        // a lane per box of 16 keys; the pages of a tile are looked up a tile ahead
        auto cell_of = [&](int t) {
          const int key = t * CW_KT + 16 * lane;
          if (lane >= CW_KT / 16 || key >= walk.s.keys) return -1;
          const int page = __ldg(table + (key >> p.page_shift));
          if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) return -1;
          return ((page * p.Hkv + r.head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        };
        int ahead = cell_of(r.t0);
        // the first two tiles need no query: they are on their way before the queries are in place
        bool ok = true;
        for (int t = r.t0; t < r.t1; ++t) {
          const int pipe = (t - r.t0) & 1, use = used[pipe] + ((t - r.t0) >> 1);
          const int cell = ahead;
          if (t + 1 < r.t1) ahead = cell_of(t + 1);
          if (t == r.t0 + 2) cw_sync(0, CW_THREADS);
          if (ok && use > 0) ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kKEmpty), use - 1));
          if (!ok) continue;
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, cell >= 0));
          if (lane == 0) mbar_arrive_expect_tx(bar(pipe, kKFull), boxes * 16 * CA_D);
          __syncwarp();
          if (cell >= 0) tma_load_2d(smem + L::kOffK + pipe * CW_HALF + lane * 16 * CA_D, &tmK, bar(pipe, kKFull), 0, cell);
          issued[pipe] = use + 1;
        }
        if (r.t1 - r.t0 <= 2) cw_sync(0, CW_THREADS);
        used[0] += (r.t1 - r.t0 + 1) / 2;
        used[1] += (r.t1 - r.t0) / 2;
        if (cw_vote(0, CW_THREADS, (bad & 4) != 0)) break;
      }
      // every copy has landed before the shared memory goes away
      if (lane == 0)
        for (int pipe = 0; pipe < 2; ++pipe)
          if (issued[pipe] > 0)
            mbar_wait_bounded(bar(pipe, kKFull), static_cast<uint32_t>((issued[pipe] - 1) & 1), nullptr, CA_WAIT_NS);
    } else {
      // -------------------------------------------------------------- products
      const uint32_t qa = smem_addr(smem + L::kOffQ);
      while (walk.next(p, &r, bad)) {
        if (walk.s.keys == 0) continue;
        cw_sync(0, CW_THREADS);
        tc_fence_after();
        if (lane == 0) {
          const int tiles = r.t1 - r.t0;
          auto logits = [&](int n) {  // S of tile n of the run
            const int pipe = n & 1, use = used[pipe] + (n >> 1);
            if (!wait(bar(pipe, kKFull), use)) return false;
            tc_fence_after();
            const uint32_t kb = smem_addr(smem + L::kOffK + pipe * CW_HALF);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_i8(tmem + pipe * 128, smem_desc_k_sw128(qa + k * 32), smem_desc_k_sw128(kb + k * 32), CW_IDESC_S,
                     k > 0 ? 1u : 0u);
            mma_commit(bar(pipe, kSFull));
            mma_commit(bar(pipe, kKEmpty));
            return true;
          };
          bool ok = logits(0);
          if (ok && tiles > 1) ok = logits(1);
          // a step of tile n: the pipeline's next S before the last P V of a tile: its softmax waits for it, and for this
          // P V only after that
          auto values = [&](int n, int step) {
            const int pipe = n & 1, use = used[pipe] + (n >> 1);
            if (step == STEPS - 1 && n + 2 < tiles && !(wait(bar(pipe, kSEmpty), use) && logits(n + 2))) return false;
            if (!wait(bar(pipe, kPFull + step), use) || (step == 0 && !wait(bar(pipe, kVFull), use))) return false;
            tc_fence_after();
            const uint32_t pa = smem_addr(smem + L::kOffP + pipe * 2 * CW_HALF);
            const uint32_t va = smem_addr(smem + L::kOffV + pipe * 2 * CW_HALF);
            // 16 keys an instruction: P's K-major rows advance 32 bytes inside a 64-key half; the values' atoms are
            // 8 keys x 64 channels (1 KB apart along the keys, the second 64 channels 16 KB on)
#pragma unroll
            for (int h = 0; h < 2; ++h)  // halves of the keys, or a step's weights and their rest
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16(tmem + 256 + pipe * 128, smem_desc_k_sw128(pa + h * CW_HALF + k * 32),
                         smem_desc_mn_sw128(va + (4 * (STEPS == 1 ? h : step) + k) * 2048, CW_HALF, 1024), CW_IDESC_O,
                         (n >= 2 || step > 0 || h > 0 || k > 0) ? 1u : 0u);
            mma_commit(bar(pipe, kODone + step));
            return true;
          };
          // both pipelines' first steps, then both their second ones, as their softmax takes turns
          for (int n = 0; n < tiles && ok; n += 2)
            for (int step = 0; step < STEPS && ok; ++step) {
              ok = values(n, step);
              if (ok && n + 1 < tiles) ok = values(n + 1, step);
            }
        }
        used[0] += (r.t1 - r.t0 + 1) / 2;
        used[1] += (r.t1 - r.t0) / 2;
        if (cw_vote(0, CW_THREADS, (bad & 4) != 0)) break;
      }
      if (lane == 0) {
        // every product issued has finished before TMEM is released
        mma_commit(drain);
        mbar_wait_bounded(drain, 0u, nullptr, CA_WAIT_NS);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncwarp();
  const int any_bad = __syncthreads_or(bad & CA_BAD), late = __syncthreads_or(bad & 4);  // a timeout is 5
  if (tid == 0) p.piece_status[blockIdx.x] = late ? CA_LATE : any_bad ? CA_BAD : 0;
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 cw_encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

template <bool F16>
cudaError_t cw_launch(const CUtensorMap& tk, const CaParams& p, cudaStream_t s) {
  static std::atomic<int> ready[64];  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (!known || ready[dev].load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(cache_attention_wide_kernel<F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             CwSmem::kAlloc);
    if (e != cudaSuccess) return e;
    if (known) ready[dev].store(1, std::memory_order_release);
  }
  cache_attention_wide_kernel<F16><<<p.workers, CW_THREADS, CwSmem::kAlloc, s>>>(tk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_wide(const CaParams& p, bool f16, int64_t cells, cudaStream_t stream) {
  const auto enc = cw_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  // key codes as rows of 128 bytes, boxes of 16 keys, 128-byte swizzle
  const cuuint64_t dims[2] = {CA_D, static_cast<cuuint64_t>(cells)};
  const cuuint64_t strides[1] = {CA_D};
  const cuuint32_t box[2] = {CA_D, 16};
  const cuuint32_t step[2] = {1, 1};
  CUtensorMap tk;
  if (enc(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p.k_codes), dims, strides, box, step,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return f16 ? cw_launch<true>(tk, p, stream) : cw_launch<false>(tk, p, stream);
}

}  // namespace convrot
