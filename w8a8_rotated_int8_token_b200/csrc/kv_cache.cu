// The rotated int8 key/value cache: written (convrot_cache_append) and read
// back (convrot_cache_read).
//
// A cell is one token of one head: 128 int8 codes c = rne(x R / s) and one
// float32 scale s = absmax(x R) / 127, R = H_128 / sqrt(128): the linear layer's
// per-token rule over a head vector, to the same bits as convrot_quant_act with
// g = 128. Reading gives (c s) R, since R is its own inverse.
//
// Bound by memory: 256 bytes on the dense side and 132 in the cell per vector.
// Four lanes share a key and its value, 32 channels each; every access on the dense
// side is 16 bytes a lane in runs of 64 per vector, and both vectors' loads are issued
// before either is transformed. Writing, five of the seven butterfly stages stay in
// registers, packed two to an instruction, and two cross lanes (64 shuffles a lane
// and vector; with 16 lanes it would be twice as many per vector).
// Reading transforms whole numbers, exact in any order, so there the tensor cores
// take five stages at once (a product with the 32-point signs, eight instructions for
// eight vectors) and nothing crosses lanes: 32768 scattered tokens of 8 heads in 36.3 us
// (204 MB, 87 % of the copy bandwidth; the scales of scattered cells cost a 32-byte
// sector each, 17 MB more) against 40.9 with the stages of writing, where shuffles and
// narrow loads kept the first-level data path 85 % busy, 47.3 with a thread per vector
// and 53.9 with the first four stages in pairs of fp16.

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"

namespace convrot {

namespace {

constexpr int kCellThreads = 64;
constexpr int kCellDim = 128;
constexpr int kBadSlot = CONVROT_ERR_INVALID_ARG;

struct CellParams {
  uint16_t* k;               // dense keys and values, [T, H, 128] with strides
  uint16_t* v;
  int64_t kt, kh, vt, vh;
  const int32_t* slots;
  int8_t* k_codes;           // [P, H, page, 128]
  int8_t* v_codes;
  float* k_scale;            // [P, H, page]
  float* v_scale;
  int pairs;                 // T H
  int H, page_shift;
  int capacity;              // P * page
  int* status;
};

// The key and the value of a thread: token t, head h; their cell, or -1.
struct CellPlace {
  int64_t t, cell;
  int h;
};

__device__ __forceinline__ CellPlace cell_place(const CellParams& p, int pair) {
  CellPlace c;
  const uint32_t t = static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.H);
  c.t = t;
  c.h = pair - static_cast<int>(t) * p.H;
  const int slot = __ldg(p.slots + t);
  c.cell = -1;
  if (slot >= 0 && slot < p.capacity) {
    const int page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    c.cell = ((static_cast<int64_t>(page) * p.H + c.h) << p.page_shift) + off;
  } else if (slot >= p.capacity && p.status != nullptr) {
    atomicOr(p.status, kBadSlot);
  }
  return c;
}

// A vector's four 16-byte pieces of a lane (channels 32 j + 8 l .. + 7) into its cell.
template <bool F16>
__device__ __forceinline__ void write_cell(const uint4 (&w)[4], int l, int64_t cell, int8_t* codes, float* scales) {
  float2 v[16];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t a[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
    const uint32_t b[4] = {w[2 + j].x, w[2 + j].y, w[2 + j].z, w[2 + j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      fwht::fwht_first_pair<F16>(a[e], fwht::widen_pair<F16>(b[e]), v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
  }
  fwht::fwht128_quad(v, l);
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m[i] = fwht::fmax3f(fabsf(v[2 * i].x), fabsf(v[2 * i].y), fmaxf(fabsf(v[2 * i + 1].x), fabsf(v[2 * i + 1].y)));
  float amax = fwht::fmax3f(fwht::fmax3f(m[0], m[1], m[2]), fwht::fmax3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  if (cell < 0) return;
  const fwht::CodeFactor f = fwht::code_factor(amax);
  const float2 ci = make_float2(f.ci, f.ci), magic = make_float2(fwht::kRoundMagic, fwht::kRoundMagic);
  const float2 pre = make_float2(f.pre, f.pre);
  int8_t* dst = codes + cell * kCellDim + 8 * l;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float2 r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = __ffma2_rn(__fmul2_rn(v[8 * j + e], pre), ci, magic);
    *reinterpret_cast<uint2*>(dst + 32 * j) =
        make_uint2(fwht::pack4(r[0].x, r[1].x, r[2].x, r[3].x), fwht::pack4(r[4].x, r[5].x, r[6].x, r[7].x));
    *reinterpret_cast<uint2*>(dst + 64 + 32 * j) =
        make_uint2(fwht::pack4(r[0].y, r[1].y, r[2].y, r[3].y), fwht::pack4(r[4].y, r[5].y, r[6].y, r[7].y));
  }
  if (l == 0) scales[cell] = fwht::scale_of<128>(amax);
}

template <bool F16>
__global__ void __launch_bounds__(kCellThreads) cache_append_kernel(const CellParams p) {
  const int pair = (blockIdx.x * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  CellPlace c{};
  c.cell = -1;
  uint4 k[4], v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = v[j] = make_uint4(0u, 0u, 0u, 0u);
  if (pair < p.pairs) {
    c = cell_place(p, pair);
    const uint16_t* kf = p.k + c.t * p.kt + c.h * p.kh + 8 * l;
    const uint16_t* vf = p.v + c.t * p.vt + c.h * p.vh + 8 * l;
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = __ldg(reinterpret_cast<const uint4*>(kf + 32 * j));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(vf + 32 * j));
  }
  write_cell<F16>(k, l, c.cell, p.k_codes, p.k_scale);
  write_cell<F16>(v, l, c.cell, p.v_codes, p.v_scale);
}

// Sums of 32 codes of 16 rows with signs, added to the bits of a float: exact.
__device__ __forceinline__ void mma_codes(uint32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, uint32_t c) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c));
}

// The signs of the 32-point transform as the operand of mma_codes: lane 4 g + t needs rows 8 t + 4 h + e (byte e of
// word h) of column 8 (g / 2) + 2 n + g % 2, so that lane t of a vector brings channels 8 t .. + 7 of a block of 32
// and gets their sums back. Of n that leaves its low bit to the word, sign[n % 2], and its high bit to an inversion
// of the second half's rows (h = 1), sign[2 + n % 2].
__device__ __forceinline__ void block_signs(int lane, uint32_t (&sign)[4]) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t flip = (__popc(t & (g >> 1)) & 1) != 0 ? 0xFEFEFEFEu : 0u;  // 1 and -1 change places
  // bytes 0 .. 3 of columns 0 .. 3 (mod 4)
  sign[0] = ((g & 1) != 0 ? 0xFF01FF01u : 0x01010101u) ^ flip;
  sign[1] = ((g & 1) != 0 ? 0x01FFFF01u : 0xFFFF0101u) ^ flip;
  sign[2] = sign[0] ^ 0xFEFEFEFEu;
  sign[3] = sign[1] ^ 0xFEFEFEFEu;
}

// A vector's four 8-byte pieces of codes (channels 32 j + 8 l .. + 7) to the same channels of the vector; zeros where
// there is no cell. The sums of 128 codes are whole numbers and every step is exact: the stages on index bits
// 0 to 4 are the matrix product, those on 5 and 6 in registers.
template <bool F16>
__device__ __forceinline__ void read_cell(const uint2 (&w)[4], const uint32_t (&sign)[4], float scale, bool there,
                                          bool any, uint16_t* dst) {
  constexpr uint32_t kBits = 0x4B400000u;  // 1.5 * 2^23: plus a sum as an integer it is that plus the sum as a float
  const float2 bias = make_float2(-12582912.0f, -12582912.0f);
  float2 v[4][4];  // channels 32 j + 8 l + 2 n, + 1 in v[j][n]
  __syncwarp();    // the products are the whole warp's, the loads and stores around them each lane's own
#pragma unroll
  for (int n = 0; n < 4; ++n) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      uint32_t d[4];
      mma_codes(d, w[j].x, w[j + 1].x, w[j].y, w[j + 1].y, sign[n & 1], sign[n], kBits);
      v[j][n] = __fadd2_rn(make_float2(__uint_as_float(d[0]), __uint_as_float(d[1])), bias);
      v[j + 1][n] = __fadd2_rn(make_float2(__uint_as_float(d[2]), __uint_as_float(d[3])), bias);
    }
  }
  const float by1 = scale * fwht::kInvSqrt128;
  const float2 by = make_float2(by1, by1);
  uint32_t out[4][4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 s0 = fwht::bfly_sum(v[0][n], v[1][n]), d0 = fwht::bfly_diff(v[0][n], v[1][n]);
    const float2 s1 = fwht::bfly_sum(v[2][n], v[3][n]), d1 = fwht::bfly_diff(v[2][n], v[3][n]);
    const float2 y[4] = {fwht::bfly_sum(s0, s1), fwht::bfly_sum(d0, d1), fwht::bfly_diff(s0, s1),
                         fwht::bfly_diff(d0, d1)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = __fmul2_rn(y[j], by);
      out[j][n] = any ? fwht::narrow_pair<F16>(x.x, x.y) : 0u;
    }
  }
  if (there) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(dst + 32 * j) = make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]);
  }
}

template <bool F16>
__global__ void __launch_bounds__(kCellThreads, 16) cache_read_kernel(const CellParams p) {
  const int pair = (blockIdx.x * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  const bool there = pair < p.pairs;
  CellPlace c{};
  c.cell = -1;
  if (there) c = cell_place(p, pair);
  uint2 k[4], v[4];
  float ks = 0.0f, vs = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = v[j] = make_uint2(0u, 0u);
  if (c.cell >= 0) {
    const int8_t* kf = p.k_codes + c.cell * kCellDim + 8 * l;
    const int8_t* vf = p.v_codes + c.cell * kCellDim + 8 * l;
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = __ldg(reinterpret_cast<const uint2*>(kf + 32 * j));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __ldg(reinterpret_cast<const uint2*>(vf + 32 * j));
    ks = __ldg(p.k_scale + c.cell);
    vs = __ldg(p.v_scale + c.cell);
  }
  uint32_t sign[4];
  block_signs(threadIdx.x & 31, sign);
  read_cell<F16>(k, sign, ks, there, c.cell >= 0, p.k + c.t * p.kt + c.h * p.kh + 8 * l);
  read_cell<F16>(v, sign, vs, there, c.cell >= 0, p.v + c.t * p.vt + c.h * p.vh + 8 * l);
}

bool aligned_to(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// The checks both directions share; CONVROT_OK with p filled in, or an error.
convrot_status cell_params(const convrot_cache_args* args, CellParams* p) {
  if (args == nullptr) return CONVROT_ERR_INVALID_ARG;
  const convrot_cache_args& a = *args;
  const convrot_cells& c = a.cells;
  if (a.dtype != CONVROT_DTYPE_BF16 && a.dtype != CONVROT_DTYPE_F16) return CONVROT_ERR_UNSUPPORTED;
  if (c.D != kCellDim) return CONVROT_ERR_UNSUPPORTED;
  if (a.T < 0 || c.H < 1 || c.num_pages < 1 || c.page_size < 1) return CONVROT_ERR_INVALID_ARG;
  if (c.page_size < CONVROT_MIN_PAGE || c.page_size > CONVROT_MAX_PAGE || (c.page_size & (c.page_size - 1)) != 0)
    return CONVROT_ERR_UNSUPPORTED;
  if (c.H > CONVROT_MAX_CACHE_HEADS || c.num_pages > 0x7FFFFFFF / c.page_size || a.T > 0x1FFFFFFF / c.H)
    return CONVROT_ERR_UNSUPPORTED;
  auto stride = [](int64_t n, int64_t st) { return n > 1 ? st : 0; };
  p->kt = stride(a.T, a.k_token), p->kh = stride(c.H, a.k_head);
  p->vt = stride(a.T, a.v_token), p->vh = stride(c.H, a.v_head);
  if ((p->kt | p->kh | p->vt | p->vh) % 8 != 0) return CONVROT_ERR_INVALID_ARG;
  if (a.T == 0) return CONVROT_OK;
  for (const void* ptr : {static_cast<const void*>(a.K), static_cast<const void*>(a.V),
                          static_cast<const void*>(c.k_codes), static_cast<const void*>(c.v_codes),
                          static_cast<const void*>(c.k_scale), static_cast<const void*>(c.v_scale)})
    if (ptr == nullptr || !aligned_to(ptr, 16)) return CONVROT_ERR_INVALID_ARG;
  if (a.slots == nullptr || !aligned_to(a.slots, 4) || !aligned_to(a.status, 4)) return CONVROT_ERR_INVALID_ARG;
  p->k = static_cast<uint16_t*>(a.K);
  p->v = static_cast<uint16_t*>(a.V);
  p->slots = a.slots;
  p->k_codes = c.k_codes;
  p->v_codes = c.v_codes;
  p->k_scale = c.k_scale;
  p->v_scale = c.v_scale;
  p->pairs = static_cast<int>(a.T * c.H);
  p->H = static_cast<int>(c.H);
  p->page_shift = 0;
  while ((int64_t{1} << p->page_shift) < c.page_size) ++p->page_shift;
  p->capacity = static_cast<int>(c.num_pages * c.page_size);
  p->status = a.status;
  return CONVROT_OK;
}

unsigned cell_grid(const CellParams& p) {
  return (static_cast<unsigned>(p.pairs) * 4 + kCellThreads - 1) / kCellThreads;
}

}  // namespace

}  // namespace convrot

extern "C" {

convrot_status convrot_cache_append(const convrot_cache_args* args, convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(args, &p);
  if (st != CONVROT_OK || args->T == 0) return st;
  (args->dtype == CONVROT_DTYPE_F16 ? cache_append_kernel<true> : cache_append_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

convrot_status convrot_cache_read(const convrot_cache_args* args, convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(args, &p);
  if (st != CONVROT_OK || args->T == 0) return st;
  (args->dtype == CONVROT_DTYPE_F16 ? cache_read_kernel<true> : cache_read_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

}  // extern "C"
