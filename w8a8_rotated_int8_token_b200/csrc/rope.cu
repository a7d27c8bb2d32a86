// Rotary positions with several axes: pairs of channels of every head vector
// turned by the angle pos[axis(i)] * freq(i) of pair i.
//
//   (y1, y2) = (x1 cos - x2 sin, x2 cos + x1 sin),
//
// the pair being channels (i, i + R/2) or, interleaved, (2i, 2i + 1); channels
// from R on are copied. The inverse turns by -angle: the transpose of the
// rotation, so it is also the gradient. The angle is a float64 product reduced
// to one turn before anything is rounded to float32 (positions in the 100000s
// would otherwise lose the angle's fraction); sine, cosine and the two products
// are float32 and the output is rounded once.
//
// Bound by memory: 2 bytes read and 2 written per channel. A CTA owns a few
// tokens; hp x (D/16) threads share a token, and a thread keeps the same eight
// pairs for every head it visits, so their sines and cosines are read from
// shared memory once. The first four heads' loads are issued before the angles
// are computed. Six CTAs of 128 threads per SM (80 registers): 43.9 us of device time
// for 16896 tokens of 32 heads (a call alone 47), 98 % of the copy bandwidth; CTAs of 256
// threads took 46.2 to 53.8 us, two heads ahead 49.5.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "convrot.h"
#include "fwht128.cuh"

namespace convrot {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;        // heads whose loads a thread has in flight
constexpr int kRopeMaxDim = 512;
constexpr int kRopeSms = 148;         // of a B200
constexpr int kRopeTableMax = 2048;   // sine/cosine pairs a CTA holds (16 KB)
constexpr float kRopeLeft = 2.0f;     // for a cosine: the pair is not turned

struct RopeParams {
  const uint16_t* x;
  uint16_t* y;
  int64_t tokens;            // B * S
  int S, H, D, R;
  int64_t xb, xs, xh, yb, ys, yh;
  const void* pos;
  int pos_float, axes;
  int64_t pa, pb, ps;
  const double* freq;
  const int32_t* axis;
  int interleaved, inverse;
  int hp;                    // heads a token's threads visit at once
  int tok;                   // tokens of a CTA
};

// (cos, sin) of pair i at token n; kRopeLeft for a pair whose axis is out of [0, axes). Such a pair is copied: turned by
// an angle of 0 an infinite channel would make its partner NaN.
__device__ __forceinline__ float2 rope_turn(const RopeParams& p, int64_t n, int i) {
  const int a = __ldg(p.axis + i);
  if (a < 0 || a >= p.axes) return make_float2(kRopeLeft, 0.0f);
  const uint32_t b = static_cast<uint32_t>(n) / static_cast<uint32_t>(p.S);  // tokens < 2^31
  const int64_t at = a * p.pa + b * p.pb + (n - static_cast<int64_t>(b) * p.S) * p.ps;
  const double pos = p.pos_float ? static_cast<double>(__ldg(static_cast<const float*>(p.pos) + at))
                                 : static_cast<double>(__ldg(static_cast<const int32_t*>(p.pos) + at));
  const double turns = pos * (__ldg(p.freq + i) * 0.15915494309189533577);
  const float r = static_cast<float>(turns - rint(turns));
  float s, c;
  sincospif(2.0f * r, &s, &c);
  return make_float2(c, p.inverse ? -s : s);
}

// Sixteen channels of a head, two runs of eight: the first and the second channels of eight pairs, or,
// interleaved, four pairs each.
template <bool F16, bool INTER>
__device__ __forceinline__ void rope_apply(uint4& lo, uint4& hi, const float2 (&cs)[8], bool turn_lo, bool turn_hi) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = fwht::widen_pair<F16>(a[i]), v = fwht::widen_pair<F16>(b[i]);
      const uint32_t x = fwht::narrow_pair<F16>(fmaf(u.x, cs[i].x, -u.y * cs[i].y), fmaf(u.y, cs[i].x, u.x * cs[i].y));
      const uint32_t y =
          fwht::narrow_pair<F16>(fmaf(v.x, cs[4 + i].x, -v.y * cs[4 + i].y), fmaf(v.y, cs[4 + i].x, v.x * cs[4 + i].y));
      a[i] = turn_lo ? x : a[i];
      b[i] = turn_hi ? y : b[i];
    }
  } else if (turn_lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = fwht::widen_pair<F16>(a[i]), v = fwht::widen_pair<F16>(b[i]);
      const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
      a[i] = fwht::narrow_pair<F16>(fmaf(u.x, c0.x, -v.x * c0.y), fmaf(u.y, c1.x, -v.y * c1.y));
      b[i] = fwht::narrow_pair<F16>(fmaf(v.x, c0.x, u.x * c0.y), fmaf(v.y, c1.x, u.y * c1.y));
    }
  }
}

// Puts the channels of the pairs in `left` back to what they were before rope_apply.
template <bool INTER>
__device__ __forceinline__ void rope_keep(uint4& lo, uint4& hi, const uint4& was_lo, const uint4& was_hi, uint32_t left) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
  const uint32_t u[4] = {was_lo.x, was_lo.y, was_lo.z, was_lo.w}, v[4] = {was_hi.x, was_hi.y, was_hi.z, was_hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t split = (left >> (2 * i) & 1u ? 0xFFFFu : 0u) | (left >> (2 * i + 1) & 1u ? 0xFFFF0000u : 0u);
    const uint32_t m = INTER ? 0u - (left >> i & 1u) : split, n = INTER ? 0u - (left >> (4 + i) & 1u) : split;
    a[i] = (a[i] & ~m) | (u[i] & m);
    b[i] = (b[i] & ~n) | (v[i] & n);
  }
}

// Sixteen-byte accesses: D and R multiples of 16, pointers and strides of 16 bytes.
template <bool F16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_kernel(const RopeParams p) {
  __shared__ float2 table[kRopeTableMax];
  const int per_head = p.D >> 4, pairs = p.R >> 1;
  const int group = p.hp * per_head;  // threads of a token
  const int slot = threadIdx.x / group, q = threadIdx.x - slot * group;
  const int h0 = q / per_head, c = q - h0 * per_head;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tok;
  const int64_t n = first + slot;
  const bool mine = slot < p.tok && n < p.tokens;
  // Channels of the thread's two runs of eight. Neighbouring threads take neighbouring runs, also of interleaved
  // pairs: with sixteen channels in a row per thread 4224 tokens of 32 heads took
  // 16.8 us for 14.1.
  const bool split = !INTER && 8 * c < pairs;
  const int d_lo = INTER || split ? 8 * c : 16 * c;
  const int d_hi = INTER ? (p.D >> 1) + 8 * c : split ? pairs + 8 * c : d_lo + 8;
  const bool turn_lo = INTER ? d_lo < p.R : split, turn_hi = INTER ? d_hi < p.R : split;
  const int pair_lo = INTER ? d_lo >> 1 : 8 * c, pair_hi = INTER ? d_hi >> 1 : 8 * c + 4;  // of four each
  const int64_t b = mine ? static_cast<uint32_t>(n) / static_cast<uint32_t>(p.S) : 0, s = mine ? n - b * p.S : 0;
  const uint16_t* x = p.x + b * p.xb + s * p.xs;
  uint16_t* y = p.y + b * p.yb + s * p.ys;

  uint4 lo[kRopeAhead], hi[kRopeAhead];
#pragma unroll
  for (int k = 0; k < kRopeAhead; ++k) {
    const int h = h0 + k * p.hp;
    if (mine && h < p.H) {
      lo[k] = *reinterpret_cast<const uint4*>(x + h * p.xh + d_lo);
      hi[k] = *reinterpret_cast<const uint4*>(x + h * p.xh + d_hi);
    }
  }
  for (int i = threadIdx.x; i < p.tok * pairs; i += kRopeThreads) {
    const int64_t at = first + i / pairs;
    if (at < p.tokens) table[i] = rope_turn(p, at, i % pairs);
  }
  __syncthreads();
  if (!mine) return;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = turn_lo ? table[slot * pairs + pair_lo + i] : make_float2(1.0f, 0.0f);
    cs[4 + i] = turn_hi ? table[slot * pairs + pair_hi + i] : make_float2(1.0f, 0.0f);
  }
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) left |= cs[i].x == kRopeLeft ? 1u << i : 0u;
  // in a loop of its own, so that the usual one has no register more: together 50.1 against 47.1 us a call for 16896
  // tokens
  auto visit = [&](auto keeps_pairs) {
    constexpr bool keeps = decltype(keeps_pairs)::value;
    for (int hb = h0; hb < p.H; hb += kRopeAhead * p.hp) {
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        const int h = hb + k * p.hp;
        if (h < p.H) {
          if (keeps) {
            const uint4 was_lo = lo[k], was_hi = hi[k];
            rope_apply<F16, INTER>(lo[k], hi[k], cs, turn_lo, turn_hi);
            rope_keep<INTER>(lo[k], hi[k], was_lo, was_hi, left);
          } else {
            rope_apply<F16, INTER>(lo[k], hi[k], cs, turn_lo, turn_hi);
          }
          *reinterpret_cast<uint4*>(y + h * p.yh + d_lo) = lo[k];
          *reinterpret_cast<uint4*>(y + h * p.yh + d_hi) = hi[k];
        }
      }
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        const int h = hb + (kRopeAhead + k) * p.hp;
        if (h < p.H) {
          lo[k] = *reinterpret_cast<const uint4*>(x + h * p.xh + d_lo);
          hi[k] = *reinterpret_cast<const uint4*>(x + h * p.xh + d_hi);
        }
      }
    }
  };
  if (left != 0) visit(std::true_type{});
  else visit(std::false_type{});
}

// Any even R, any strides and alignment of 2 bytes: one CTA per token, one pair
// (or one copied channel) per thread and step.
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(const RopeParams p) {
  __shared__ float2 table[kRopeMaxDim / 2];
  const int pairs = p.R >> 1, steps = p.D - pairs;  // pairs, then the channels that are copied
  const int64_t n = blockIdx.x, b = n / p.S, s = n - b * p.S;
  const uint16_t* x = p.x + b * p.xb + s * p.xs;
  uint16_t* y = p.y + b * p.yb + s * p.ys;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) table[i] = rope_turn(p, n, i);
  __syncthreads();
  const int64_t work = static_cast<int64_t>(p.H) * steps;
  for (int64_t w = threadIdx.x; w < work; w += kRopeThreads) {
    const int64_t h = w / steps;
    const int i = static_cast<int>(w - h * steps);
    if (i < pairs) {
      const int d1 = p.interleaved ? 2 * i : i, d2 = p.interleaved ? 2 * i + 1 : i + pairs;
      const uint32_t w = x[h * p.xh + d1] | static_cast<uint32_t>(x[h * p.xh + d2]) << 16;
      const float2 u = fwht::widen_pair<F16>(w);
      const float2 cs = table[i];
      const uint32_t o = cs.x == kRopeLeft
                             ? w
                             : fwht::narrow_pair<F16>(fmaf(u.x, cs.x, -u.y * cs.y), fmaf(u.y, cs.x, u.x * cs.y));
      y[h * p.yh + d1] = static_cast<uint16_t>(o);
      y[h * p.yh + d2] = static_cast<uint16_t>(o >> 16);
    } else {
      y[h * p.yh + pairs + i] = x[h * p.xh + pairs + i];
    }
  }
}

}  // namespace

}  // namespace convrot

extern "C" {

convrot_status convrot_rope(const convrot_rope_args* args, convrot_stream_t stream) {
  using namespace convrot;
  if (args == nullptr) return CONVROT_ERR_INVALID_ARG;
  const convrot_rope_args& a = *args;
  if ((a.dtype != CONVROT_DTYPE_BF16 && a.dtype != CONVROT_DTYPE_F16) ||
      (a.pos_dtype != CONVROT_POS_I32 && a.pos_dtype != CONVROT_POS_F32))
    return CONVROT_ERR_UNSUPPORTED;
  if (a.B < 0 || a.S < 0 || a.H < 1 || a.D < 1 || a.R < 0 || a.R > a.D || a.R % 2 != 0 || a.axes < 1)
    return CONVROT_ERR_INVALID_ARG;
  if (a.D > kRopeMaxDim || a.H > 65535 || a.B > 0x7FFFFFFF || a.S > 0x7FFFFFFF || a.axes > 0x7FFFFFFF ||
      (a.S > 0 && a.B > 0x7FFFFFFF / a.S))
    return CONVROT_ERR_UNSUPPORTED;
  if (a.B == 0 || a.S == 0) return CONVROT_OK;  // no tokens
  if (a.X == nullptr || a.Y == nullptr ||
      (a.R > 0 && (a.positions == nullptr || a.freq == nullptr || a.axis == nullptr)))
    return CONVROT_ERR_INVALID_ARG;
  auto aligned = [](const void* ptr, uintptr_t to) { return (reinterpret_cast<uintptr_t>(ptr) % to) == 0; };
  if (!aligned(a.X, 2) || !aligned(a.Y, 2) || !aligned(a.positions, 4) || !aligned(a.freq, 8) || !aligned(a.axis, 4))
    return CONVROT_ERR_INVALID_ARG;
  auto stride = [](int64_t n, int64_t st) { return n > 1 ? st : 0; };
  RopeParams p{};
  p.x = static_cast<const uint16_t*>(a.X);
  p.y = static_cast<uint16_t*>(a.Y);
  p.tokens = a.B * a.S;
  p.S = static_cast<int>(a.S);
  p.H = static_cast<int>(a.H);
  p.D = static_cast<int>(a.D);
  p.R = static_cast<int>(a.R);
  p.xb = stride(a.B, a.x_batch), p.xs = stride(a.S, a.x_token), p.xh = stride(a.H, a.x_head);
  p.yb = stride(a.B, a.y_batch), p.ys = stride(a.S, a.y_token), p.yh = stride(a.H, a.y_head);
  p.pos = a.positions;
  p.pos_float = a.pos_dtype == CONVROT_POS_F32;
  p.axes = static_cast<int>(a.axes);
  p.pa = stride(a.axes, a.pos_axis), p.pb = stride(a.B, a.pos_batch), p.ps = stride(a.S, a.pos_token);
  p.freq = a.freq;
  p.axis = a.axis;
  p.interleaved = a.interleaved != 0;
  p.inverse = a.inverse != 0;
  const bool f16 = a.dtype == CONVROT_DTYPE_F16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t strides = p.xb | p.xs | p.xh | p.yb | p.ys | p.yh;
  if (p.D % 16 != 0 || p.R % 16 != 0 || strides % 8 != 0 || !aligned(p.x, 16) || !aligned(p.y, 16)) {
    (f16 ? rope_scalar_kernel<true> : rope_scalar_kernel<false>)<<<static_cast<unsigned>(p.tokens), kRopeThreads, 0,
                                                                    s>>>(p);
    return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
  }
  // A quarter of the heads at once gives each thread kRopeAhead loads in flight;
  // few tokens take all threads for each, since only latency counts.
  const int per_head = p.D / 16, most = kRopeThreads / per_head;
  const bool few = p.tokens <= 1024;
  p.hp = few ? p.H : (p.H + kRopeAhead - 1) / kRopeAhead;
  if (p.hp > most) p.hp = most;
  p.tok = kRopeThreads / (p.hp * per_head);
  if (p.R > 0 && p.tok > kRopeTableMax / (p.R / 2)) p.tok = kRopeTableMax / (p.R / 2);
  const int64_t spread = (p.tokens + kRopeSms - 1) / kRopeSms;  // a CTA on every SM
  if (few && p.tok > spread) p.tok = static_cast<int>(spread);
  const unsigned grid = static_cast<unsigned>((p.tokens + p.tok - 1) / p.tok);
  if (p.interleaved)
    (f16 ? rope_kernel<true, true> : rope_kernel<false, true>)<<<grid, kRopeThreads, 0, s>>>(p);
  else
    (f16 ? rope_kernel<true, false> : rope_kernel<false, false>)<<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

}  // extern "C"
