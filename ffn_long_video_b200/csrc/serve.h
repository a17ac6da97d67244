// What the calls around the key-value cache share: rotary positions (rope.cu),
// the page plan (kv_plan.cu) and attention of one new token (decode_attn.cu).
#pragma once

#include "common.cuh"
#include "host_util.h"

namespace adaspark {

// Rows of heads: element (t, h, e) at t * ts + h * hs + e (strides in elements).
struct HeadRows {
  int64_t ts, hs;
};

// A paged cache: element (page, offset, head, e) at page * ps + offset * ts + head * hs + e.
struct CacheRows {
  int64_t ps, ts, hs;
  int32_t n_pages, page_size;
};

inline size_t elem_size(int dtype) { return dtype == ADASPARK_BF16 ? 2 : 4; }

// The kernels move 16 bytes at a time: a 16-byte base and strides of whole 16 bytes.
inline bool rows_aligned(const void* base, int64_t ts, int64_t hs, int dtype) {
  const int64_t per16 = 16 / (int64_t)elem_size(dtype);
  return aligned(base, 16) && ts % per16 == 0 && hs % per16 == 0;
}

// No two of the n x h rows of d elements share memory (rows that are written).
inline bool rows_distinct(int64_t n, int64_t h, int64_t d, int64_t ts, int64_t hs) {
  if (h > 1 && hs < d) return false;
  if (n > 1 && ts < d) return false;
  if (h <= 1 || n <= 1) return true;
  return ts >= (h - 1) * hs + d || hs >= (n - 1) * ts + d;
}

inline bool head_sizes_ok(int hq, int hkv, int d, int dtype) {
  if (dtype != ADASPARK_BF16 && dtype != ADASPARK_FP32) return false;
  return hq >= 1 && hkv >= 1 && hq <= 4096 && hq % hkv == 0 && (d == 64 || d == 128);
}

// A cache the kernels can address: slots in 31 bits, aligned rows that do not
// share memory, pages apart (tokens and heads of a page in either order).
inline bool cache_ok(const void* k, const void* v, const CacheRows& c, int hkv, int d, int dtype) {
  if (!k || !v || c.n_pages < 1 || c.page_size < 1) return false;
  if ((int64_t)c.n_pages * c.page_size > INT32_MAX) return false;
  const int64_t per16 = 16 / (int64_t)elem_size(dtype);
  if (!aligned(k, 16) || !aligned(v, 16) || c.ps % per16 || c.ts % per16 || c.hs % per16)
    return false;
  if (!rows_distinct(c.page_size, hkv, d, c.ts, c.hs)) return false;
  const int64_t page_span = (int64_t)(c.page_size - 1) * c.ts + (int64_t)(hkv - 1) * c.hs + d;
  return c.n_pages == 1 || c.ps >= page_span;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? ADASPARK_OK : ADASPARK_ECUDA; }

// Eight consecutive elements as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

}  // namespace adaspark
