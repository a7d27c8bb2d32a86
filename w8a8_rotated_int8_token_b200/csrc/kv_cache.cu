// The rotated int8 key/value cache: written (convrot_cache_append) and read
// back (convrot_cache_read).
//
// A cell is one token of one head: 128 int8 codes c = rne(x R / s) and one
// float32 scale s = absmax(x R) / 127, R = H_128 / sqrt(128): the linear layer's
// per-token rule over a head vector, to the same bits as convrot_quant_act with
// g = 128. Reading gives (c s) R, since R is its own inverse.
//
// Bound by memory: 256 bytes on the dense side and 132 in the cell per vector.
// Four lanes share a vector, 32 channels each: five of the seven butterfly
// stages stay in registers and two cross lanes (64 shuffles a lane; with 16
// lanes a vector it would be twice the shuffles per vector), and every access
// is 16 bytes a lane on the dense side with 64-byte runs per vector.

#include <cuda_runtime.h>

#include <cstdint>

#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"

namespace convrot {

namespace {

constexpr int kCellThreads = 128;
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
  int64_t vectors;           // 2 T H
  int H, page_shift;
  int capacity;              // P * page
  int* status;
};

// The vector of a thread: token t, head h, keys or values; its cell, or -1.
struct CellPlace {
  int64_t t;
  int h;
  bool value;
  int64_t cell;
};

__device__ __forceinline__ CellPlace cell_place(const CellParams& p, int64_t vec) {
  CellPlace c;
  const uint32_t two_h = 2u * static_cast<uint32_t>(p.H);
  const uint32_t t = static_cast<uint32_t>(vec) / two_h;  // vectors < 2^31
  const uint32_t rest = static_cast<uint32_t>(vec) - t * two_h;
  c.t = t;
  c.value = rest >= static_cast<uint32_t>(p.H);
  c.h = static_cast<int>(c.value ? rest - p.H : rest);
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

template <bool F16>
__global__ void __launch_bounds__(kCellThreads) cache_append_kernel(const CellParams p) {
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  const bool there = vec < p.vectors;
  CellPlace c{};
  c.cell = -1;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  if (there) {
    c = cell_place(p, vec);
    const uint16_t* src = c.value ? p.v + c.t * p.vt + c.h * p.vh : p.k + c.t * p.kt + c.h * p.kh;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * l));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = fwht::widen_pair<F16>(u[e]);
        v[8 * j + 2 * e] = f.x;
        v[8 * j + 2 * e + 1] = f.y;
      }
    }
  }
  fwht::fwht128_quad(v, l);
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m[i] = fwht::fmax3f(fabsf(v[4 * i]), fabsf(v[4 * i + 1]), fmaxf(fabsf(v[4 * i + 2]), fabsf(v[4 * i + 3])));
  float amax = fwht::fmax3f(fwht::fmax3f(m[0], m[1], m[2]), fwht::fmax3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  if (c.cell < 0) return;
  const fwht::CodeFactor f = fwht::code_factor(amax);
  int8_t* dst = (c.value ? p.v_codes : p.k_codes) + c.cell * kCellDim;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = fmaf(v[8 * j + e] * f.pre, f.ci, fwht::kRoundMagic);
    *reinterpret_cast<uint2*>(dst + 32 * j + 8 * l) =
        make_uint2(fwht::pack4(r[0], r[1], r[2], r[3]), fwht::pack4(r[4], r[5], r[6], r[7]));
  }
  if (l == 0) (c.value ? p.v_scale : p.k_scale)[c.cell] = fwht::scale_of<128>(amax);
}

template <bool F16>
__global__ void __launch_bounds__(kCellThreads) cache_read_kernel(const CellParams p) {
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  const bool there = vec < p.vectors;
  CellPlace c{};
  c.cell = -1;
  if (there) c = cell_place(p, vec);
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  float scale = 0.0f;
  if (c.cell >= 0) {
    const int8_t* src = (c.value ? p.v_codes : p.k_codes) + c.cell * kCellDim;
    scale = __ldg((c.value ? p.v_scale : p.k_scale) + c.cell) * fwht::kInvSqrt128;
    uint2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint2*>(src + 32 * j + 8 * l));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // float of a signed byte: the byte plus 128 in the low bits of 2^23, exactly
        const uint32_t u = (e < 4 ? w[j].x : w[j].y) ^ 0x80808080u;
        v[8 * j + e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + (e & 3))) - 8388736.0f;
      }
    }
  }
  fwht::fwht128_quad(v, l);  // sums of 128 codes: exact in float32
  if (!there) return;
  uint16_t* dst = c.value ? p.v + c.t * p.vt + c.h * p.vh : p.k + c.t * p.kt + c.h * p.kh;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 o;
    uint32_t* u = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = c.cell < 0 ? 0u : fwht::narrow_pair<F16>(v[8 * j + 2 * e] * scale, v[8 * j + 2 * e + 1] * scale);
    *reinterpret_cast<uint4*>(dst + 32 * j + 8 * l) = o;
  }
}

bool aligned_to(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// The checks both directions share; CONVROT_OK with p filled in, or an error.
convrot_status cell_params(const void* K, const void* V, int dtype, int64_t T, int64_t H, int64_t D, int64_t kt,
                           int64_t kh, int64_t vt, int64_t vh, const int32_t* slots, const int8_t* k_codes,
                           const int8_t* v_codes, const float* k_scale, const float* v_scale, int64_t num_pages,
                           int64_t page_size, int* status, CellParams* p) {
  if (dtype != CONVROT_DTYPE_BF16 && dtype != CONVROT_DTYPE_F16) return CONVROT_ERR_UNSUPPORTED;
  if (D != kCellDim) return CONVROT_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || num_pages < 1 || page_size < 1) return CONVROT_ERR_INVALID_ARG;
  if (page_size < CONVROT_MIN_PAGE || page_size > CONVROT_MAX_PAGE || (page_size & (page_size - 1)) != 0)
    return CONVROT_ERR_UNSUPPORTED;
  if (H > CONVROT_MAX_CACHE_HEADS || num_pages > 0x7FFFFFFF / page_size || T > 0x3FFFFFFF / H)
    return CONVROT_ERR_UNSUPPORTED;
  if (kt % 8 != 0 || kh % 8 != 0 || vt % 8 != 0 || vh % 8 != 0) return CONVROT_ERR_INVALID_ARG;
  if (T == 0) return CONVROT_OK;
  if (K == nullptr || V == nullptr || slots == nullptr || k_codes == nullptr || v_codes == nullptr ||
      k_scale == nullptr || v_scale == nullptr)
    return CONVROT_ERR_INVALID_ARG;
  if (!aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(slots, 4) || !aligned_to(k_codes, 16) ||
      !aligned_to(v_codes, 16) || !aligned_to(k_scale, 16) || !aligned_to(v_scale, 16) || !aligned_to(status, 4))
    return CONVROT_ERR_INVALID_ARG;
  p->k = const_cast<uint16_t*>(static_cast<const uint16_t*>(K));
  p->v = const_cast<uint16_t*>(static_cast<const uint16_t*>(V));
  p->kt = kt, p->kh = kh, p->vt = vt, p->vh = vh;
  p->slots = slots;
  p->k_codes = const_cast<int8_t*>(k_codes);
  p->v_codes = const_cast<int8_t*>(v_codes);
  p->k_scale = const_cast<float*>(k_scale);
  p->v_scale = const_cast<float*>(v_scale);
  p->vectors = 2 * T * H;
  p->H = static_cast<int>(H);
  p->page_shift = 0;
  while ((int64_t{1} << p->page_shift) < page_size) ++p->page_shift;
  p->capacity = static_cast<int>(num_pages * page_size);
  p->status = status;
  return CONVROT_OK;
}

unsigned cell_grid(const CellParams& p) {
  return static_cast<unsigned>((p.vectors * 4 + kCellThreads - 1) / kCellThreads);
}

}  // namespace

}  // namespace convrot

extern "C" {

convrot_status convrot_cache_append(const void* K, const void* V, int dtype, int64_t T, int64_t H, int64_t D,
                                    int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                    const int32_t* slots, int8_t* k_codes, int8_t* v_codes, float* k_scale,
                                    float* v_scale, int64_t num_pages, int64_t page_size, int* status,
                                    convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(K, V, dtype, T, H, D, k_token, k_head, v_token, v_head, slots, k_codes, v_codes,
                                        k_scale, v_scale, num_pages, page_size, status, &p);
  if (st != CONVROT_OK || T == 0) return st;
  (dtype == CONVROT_DTYPE_F16 ? cache_append_kernel<true> : cache_append_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

convrot_status convrot_cache_read(const int32_t* slots, int64_t T, int64_t H, int64_t D, const int8_t* k_codes,
                                  const int8_t* v_codes, const float* k_scale, const float* v_scale,
                                  int64_t num_pages, int64_t page_size, void* K, void* V, int dtype, int64_t k_token,
                                  int64_t k_head, int64_t v_token, int64_t v_head, int* status,
                                  convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(K, V, dtype, T, H, D, k_token, k_head, v_token, v_head, slots, k_codes, v_codes,
                                        k_scale, v_scale, num_pages, page_size, status, &p);
  if (st != CONVROT_OK || T == 0) return st;
  (dtype == CONVROT_DTYPE_F16 ? cache_read_kernel<true> : cache_read_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

}  // extern "C"
