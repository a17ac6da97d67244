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

constexpr int kMaxSeqs = 1 << 24;  // sequences of a plan or a decode call

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

// The arguments that describe norm, positions and rotation (rope.cu).
bool qk_rope_args_ok(const double* freq, int rot, int d, const int32_t* positions, int n_axes,
                     const int32_t* sections, float magnitude, const void* w_q, const void* w_k,
                     float eps);

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? ADASPARK_OK : ADASPARK_ECUDA; }

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // nothing is read for 0; the 16 bytes become zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
// 8 or 16 bytes as they are.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// V (4 or 8) consecutive elements as they lie in memory, and as fp32 pairs.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if (kWords == 2) {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      w[0] = r.x;
      w[1] = r.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = r.x;
        w[i + 1] = r.y;
        w[i + 2] = r.z;
        w[i + 3] = r.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) =
            make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[V / 2]) const {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      v[i] = sizeof(T) == 2 ? bf16x2_f2(w[i])
                            : f2(__uint_as_float(w[(2 * i) % kWords]),
                                 __uint_as_float(w[(2 * i + 1) % kWords]));
  }
  __device__ __forceinline__ void set(const F2 (&v)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = unpack(v[i]);
      if (sizeof(T) == 2) {
        w[i] = pack_bf16x2(x.x, x.y);
      } else {
        w[(2 * i) % kWords] = __float_as_uint(x.x);
        w[(2 * i + 1) % kWords] = __float_as_uint(x.y);
      }
    }
  }
};

}  // namespace adaspark
