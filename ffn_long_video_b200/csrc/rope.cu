// Rotary positions of queries and keys with their per-head RMSNorm, forward
// (optionally into a paged key-value cache) and backward.
//
// For one head x of d elements, with r = 1 / sqrt(mean(x^2) + eps) and a weight w:
//   n = x r w            (n = x without a weight)
//   pair i < rot/2 turns by the angle a = pos * freq_i, scaled by a magnitude m:
//   (n_f, n_s) -> m (n_f cos a - n_s sin a, n_s cos a + n_f sin a)
//   with (f, s) = (i, i + rot/2), or (2i, 2i + 1) interleaved;
//   elements from rot on keep n.
// Backward, g = the rotation's transpose applied to dy:
//   dw = sum over tokens and heads of g x r;  dx = r (g w - x r mean(g w x r)).
//
// Memory-bound: every element is read and written once. d/16 lanes own a head,
// two runs of 8 elements each (16-byte accesses in bf16): the runs of a rotated
// lane hold both halves of its pairs in either layout, so the rotation needs no
// exchange, and the norm's sum takes log2(d/16) shuffles. The warp's groups of
// lanes share one token's angles: each lane computes 8 / groups of them and the
// warp exchanges them by shuffles. Angles are reduced to a turn in 64 bits
// (positions of 2^20 and more keep full fp32 accuracy), sines and cosines, norms
// and rotations are in 32 bits and outputs rounded once.
#include <cmath>

#include "serve.h"

namespace adaspark {

struct RopeArgs {
  const void *q, *k, *v;
  void *qo, *ko;                 // ko may be null with a cache
  HeadRows qs, ks, vs, qos, kos;
  const int32_t* pos;            // [axes, n]
  int64_t pos_axis;              // stride between axes (0: one axis)
  const double* freq;            // [rot/2]
  const void *wq, *wk;           // [d] or null
  const int32_t* slots;          // [n]: cache slot of each token (with a cache)
  void *kc, *vc;
  CacheRows cs;
  int32_t rot, sec0, sec01;      // pairs below sec0 use axis 0, below sec01 axis 1, others 2
  int32_t n, hq, hkv, parts;
  float eps, magnitude;
};

constexpr double kInvTwoPi = 0.15915494309189533577;

template <int D>
struct RopeMap {
  static constexpr int kLanes = D / 16;          // lanes per head
  static constexpr int kHeads = 32 / kLanes;     // heads per warp step
  static constexpr int kAngles = 8 / kHeads > 0 ? 8 / kHeads : 1;  // angles a lane computes
};

// First elements of the two 8-element runs of lane `l` of a head.
__device__ __forceinline__ void rope_runs(int l, int rot, int* e0, int* e1) {
  const int rl = rot >> 4;  // rotated lanes
  if (l < rl) {
    *e0 = 8 * l;
    *e1 = 8 * l + (rot >> 1);
  } else {
    *e0 = rot + 16 * (l - rl);
    *e1 = *e0 + 8;
  }
}

// Pair index of entry e (0..7) of a rotated lane's eight pairs.
template <bool IL>
__device__ __forceinline__ int rope_pair(int l, int e, int rot) {
  if (!IL) return 8 * l + e;
  return e < 4 ? 4 * l + e : 4 * l + (rot >> 2) + (e - 4);
}

// cos and sin (times the magnitude) of a token's eight pairs for this lane;
// 1 and 0 for a lane outside the rotated part.
template <int D, bool IL>
__device__ __forceinline__ void rope_angles(const RopeArgs& a, int t, int lane, float (&c)[8],
                                            float (&s)[8]) {
  using M = RopeMap<D>;
  const int l = lane % M::kLanes, grp = lane / M::kLanes;
  const bool turns = l < (a.rot >> 4);
  float mc[M::kAngles], ms[M::kAngles];
#pragma unroll
  for (int i = 0; i < M::kAngles; ++i) {
    mc[i] = 1.f;
    ms[i] = 0.f;
    if (turns) {
      const int pair = rope_pair<IL>(l, grp * M::kAngles + i, a.rot);
      const int axis = pair < a.sec0 ? 0 : pair < a.sec01 ? 1 : 2;
      const double turn = (double)a.pos[axis * a.pos_axis + t] * a.freq[pair] * kInvTwoPi;
      float sn, cn;
      sincospif(2.f * (float)(turn - rint(turn)), &sn, &cn);
      mc[i] = cn * a.magnitude;
      ms[i] = sn * a.magnitude;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int src = (e / M::kAngles) * M::kLanes + l;
    c[e] = __shfl_sync(0xffffffffu, mc[e % M::kAngles], src);
    s[e] = __shfl_sync(0xffffffffu, ms[e % M::kAngles], src);
  }
}

// Rotates a lane's two runs in place (sign = -1 for the transpose).
template <bool IL>
__device__ __forceinline__ void rope_turn(float (&u)[8], float (&v)[8], const float (&c)[8],
                                          const float (&s)[8], float sign) {
  if (!IL) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = u[e], y = v[e], sn = sign * s[e];
      u[e] = x * c[e] - y * sn;
      v[e] = y * c[e] + x * sn;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = u[2 * e], y = u[2 * e + 1], sn = sign * s[e];
      u[2 * e] = x * c[e] - y * sn;
      u[2 * e + 1] = y * c[e] + x * sn;
      const float z = v[2 * e], w = v[2 * e + 1], sm = sign * s[4 + e];
      v[2 * e] = z * c[4 + e] - w * sm;
      v[2 * e + 1] = w * c[4 + e] + z * sm;
    }
  }
}

template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per (token, part of its heads): queries, then keys, then (with a
// cache) values, which are copied.
template <typename T, int D, bool IL, bool CACHE>
__global__ void __launch_bounds__(128) rope_kernel(const RopeArgs a) {
  using M = RopeMap<D>;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(item / a.parts), part = (int)(item % a.parts);
  if (t >= a.n) return;
  const int l = lane % M::kLanes, grp = lane / M::kLanes;
  const int heads = a.hq + a.hkv * (CACHE ? 2 : 1);
  const int steps = (heads + M::kHeads - 1) / M::kHeads;
  const int per = (steps + a.parts - 1) / a.parts;
  const int s0 = part * per, s1 = min(steps, s0 + per);
  int e0, e1;
  rope_runs(l, a.rot, &e0, &e1);
  float c[8], s[8];
  if (a.rot > 0) rope_angles<D, IL>(a, t, lane, c, s);
  const bool norm = a.wq || a.wk;
  T *kc = nullptr, *vc = nullptr;
  if (CACHE) {
    const int slot = a.slots[t];
    if (slot >= 0 && slot < a.cs.n_pages * a.cs.page_size) {
      const int64_t at = (int64_t)(slot / a.cs.page_size) * a.cs.ps +
                         (int64_t)(slot % a.cs.page_size) * a.cs.ts;
      kc = static_cast<T*>(a.kc) + at;
      vc = static_cast<T*>(a.vc) + at;
    }
  }
  for (int st = s0; st < s1; ++st) {
    const int h = st * M::kHeads + grp;
    const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
    const T* src = nullptr;
    const T* w = nullptr;
    if (is_q) {
      src = static_cast<const T*>(a.q) + t * a.qs.ts + h * a.qs.hs;
      w = static_cast<const T*>(a.wq);
    } else if (is_k) {
      src = static_cast<const T*>(a.k) + t * a.ks.ts + (h - a.hq) * a.ks.hs;
      w = static_cast<const T*>(a.wk);
    } else if (CACHE && h < heads) {
      src = static_cast<const T*>(a.v) + t * a.vs.ts + (h - a.hq - a.hkv) * a.vs.hs;
    }
    float u[8] = {}, v[8] = {};
    if (src) {
      load8(src + e0, u);
      load8(src + e1, v);
    }
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
      ss = head_sum<M::kLanes>(ss);
      if (w) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float g[8];
        load8(w + e0, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = u[e] * r * g[e];
        load8(w + e1, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * r * g[e];
      }
    }
    if ((is_q || is_k) && l < (a.rot >> 4)) rope_turn<IL>(u, v, c, s, 1.f);
    if (is_q) {
      T* o = static_cast<T*>(a.qo) + t * a.qos.ts + h * a.qos.hs;
      store8(o + e0, u);
      store8(o + e1, v);
    } else if (is_k) {
      if (a.ko) {
        T* o = static_cast<T*>(a.ko) + t * a.kos.ts + (h - a.hq) * a.kos.hs;
        store8(o + e0, u);
        store8(o + e1, v);
      }
      if (CACHE && kc) {
        store8(kc + (h - a.hq) * a.cs.hs + e0, u);
        store8(kc + (h - a.hq) * a.cs.hs + e1, v);
      }
    } else if (CACHE && src && vc) {
      store8(vc + (h - a.hq - a.hkv) * a.cs.hs + e0, u);
      store8(vc + (h - a.hq - a.hkv) * a.cs.hs + e1, v);
    }
  }
}

// Backward: warps walk tokens with a fixed stride, so the partial sums of the
// weights' gradients have a fixed order; each block writes one row of them.
// dy in T2, x in T, dx in fp32.
template <typename T, typename T2, int D, bool IL>
__global__ void __launch_bounds__(128)
    rope_bwd_kernel(const RopeArgs a, const void* dq, const void* dk, HeadRows dqs, HeadRows dks,
                    float* gq, float* gk, float* part) {
  using M = RopeMap<D>;
  __shared__ float sum[4 * M::kHeads][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % M::kLanes, grp = lane / M::kLanes;
  const int heads = a.hq + a.hkv;
  const int steps = (heads + M::kHeads - 1) / M::kHeads;
  int e0, e1;
  rope_runs(l, a.rot, &e0, &e1);
  float dwq[16] = {}, dwk[16] = {};
  const bool norm = a.wq || a.wk;
  for (int t = blockIdx.x * 4 + warp; t < a.n; t += gridDim.x * 4) {
    float c[8], s[8];
    if (a.rot > 0) rope_angles<D, IL>(a, t, lane, c, s);
    for (int st = 0; st < steps; ++st) {
      const int h = st * M::kHeads + grp;
      const bool is_q = h < a.hq, is_k = !is_q && h < heads;
      float u[8] = {}, v[8] = {};
      const T* w = nullptr;
      if (is_q) {
        const T2* p = static_cast<const T2*>(dq) + t * dqs.ts + h * dqs.hs;
        load8(p + e0, u);
        load8(p + e1, v);
        w = static_cast<const T*>(a.wq);
      } else if (is_k) {
        const T2* p = static_cast<const T2*>(dk) + t * dks.ts + (h - a.hq) * dks.hs;
        load8(p + e0, u);
        load8(p + e1, v);
        w = static_cast<const T*>(a.wk);
      }
      if (l < (a.rot >> 4)) rope_turn<IL>(u, v, c, s, -1.f);
      if (norm) {
        float x[8] = {}, y[8] = {};
        if (w) {
          const T* p = is_q ? static_cast<const T*>(a.q) + t * a.qs.ts + h * a.qs.hs
                            : static_cast<const T*>(a.k) + t * a.ks.ts + (h - a.hq) * a.ks.hs;
          load8(p + e0, x);
          load8(p + e1, y);
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
        ss = head_sum<M::kLanes>(ss);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float dot = 0.f;
        if (w) {
          float g[8];
          load8(w + e0, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= r;
            const float dw = u[e] * x[e];
            if (is_q) dwq[e] += dw; else dwk[e] += dw;
            u[e] *= g[e];
            dot = fmaf(u[e], x[e], dot);
          }
          load8(w + e1, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] *= r;
            const float dw = v[e] * y[e];
            if (is_q) dwq[8 + e] += dw; else dwk[8 + e] += dw;
            v[e] *= g[e];
            dot = fmaf(v[e], y[e], dot);
          }
        }
        dot = head_sum<M::kLanes>(dot) * (1.f / D);
        if (w) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            u[e] = r * (u[e] - x[e] * dot);
            v[e] = r * (v[e] - y[e] * dot);
          }
        }
      }
      if (is_q) {
        float* o = gq + ((int64_t)t * a.hq + h) * D;
        store8(o + e0, u);
        store8(o + e1, v);
      } else if (is_k) {
        float* o = gk + ((int64_t)t * a.hkv + (h - a.hq)) * D;
        store8(o + e0, u);
        store8(o + e1, v);
      }
    }
  }
  if (!norm) return;
  float(*mine)[D] = sum[warp * M::kHeads + grp];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mine[0][e0 + e] = dwq[e];
    mine[0][e1 + e] = dwq[8 + e];
    mine[1][e0 + e] = dwk[e];
    mine[1][e1 + e] = dwk[8 + e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 128) {
    float acc = 0.f;
#pragma unroll
    for (int g = 0; g < 4 * M::kHeads; ++g) acc += sum[g][i / D][i % D];
    part[(int64_t)blockIdx.x * 2 * D + i] = acc;
  }
}

// Sums the blocks' rows, 32 columns per block: column c of rows y, y + 32, ...
__global__ void __launch_bounds__(1024)
    rope_dw_kernel(const float* part, int rows, int d, float* dwq, float* dwk) {
  __shared__ float sum[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  float acc = 0.f;
  for (int r = y; r < rows; r += 32) acc += part[(int64_t)r * 2 * d + col];
  sum[y][x] = acc;
  __syncthreads();
  if (y == 0) {
    acc = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) acc += sum[r][x];
    float* o = col < d ? dwq : dwk;
    if (o) o[col % d] = acc;
  }
}

namespace {

constexpr int kBwdBlocksPerSm = 4;
constexpr int kBwdMaxBlocks = 148 * kBwdBlocksPerSm;

// The arguments that describe positions and rotation.
bool rope_ok(const double* freq, int rot, int d, const int32_t* positions, int n_axes,
             const int32_t* sections, float magnitude) {
  if (rot < 0 || rot > d || rot % 16 != 0) return false;
  if (rot == 0) return true;
  if (!freq || !positions || !aligned(freq, 8) || !aligned(positions, 4)) return false;
  if (!std::isfinite(magnitude)) return false;
  if (n_axes == 1) return true;
  if (n_axes != 3 || !sections) return false;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (sections[i] < 0) return false;
    sum += sections[i];
  }
  return sum == rot / 2;
}

void set_rope(RopeArgs* a, const double* freq, int rot, const int32_t* positions, int n_axes,
              const int32_t* sections, float magnitude, int n) {
  a->freq = freq;
  a->rot = rot;
  a->pos = positions;
  a->pos_axis = n_axes == 3 ? n : 0;
  a->sec0 = n_axes == 3 ? sections[0] : rot / 2;
  a->sec01 = n_axes == 3 ? sections[0] + sections[1] : rot / 2;
  a->magnitude = magnitude;
  a->n = n;
}

template <typename T, int D, bool CACHE>
cudaError_t launch_rope(RopeArgs a, bool il, int sms, cudaStream_t s) {
  const int heads = a.hq + a.hkv * (CACHE ? 2 : 1);
  const int steps = (heads + RopeMap<D>::kHeads - 1) / RopeMap<D>::kHeads;
  // few tokens: a warp per step of heads, so that a token's heads run side by side
  a.parts = (int64_t)a.n < (int64_t)sms * 16 ? steps : 1;
  const int64_t items = (int64_t)a.n * a.parts;
  const dim3 grid((unsigned)((items + 3) / 4)), block(128);
  const char* name = CACHE ? "qk_rope_append" : "qk_rope";
  if (il) return launch(name, rope_kernel<T, D, true, CACHE>, grid, block, 0, s, a);
  return launch(name, rope_kernel<T, D, false, CACHE>, grid, block, 0, s, a);
}

template <bool CACHE>
cudaError_t dispatch_rope(const RopeArgs& a, int dtype, int d, bool il, int sms, cudaStream_t s) {
  if (dtype == ADASPARK_BF16)
    return d == 128 ? launch_rope<__nv_bfloat16, 128, CACHE>(a, il, sms, s)
                    : launch_rope<__nv_bfloat16, 64, CACHE>(a, il, sms, s);
  return d == 128 ? launch_rope<float, 128, CACHE>(a, il, sms, s)
                  : launch_rope<float, 64, CACHE>(a, il, sms, s);
}

struct BwdCall {
  RopeArgs a;
  const void *dq, *dk;
  HeadRows dqs, dks;
  float *gq, *gk, *part;
  int blocks;
};

template <typename T, typename T2, int D>
cudaError_t launch_bwd(const BwdCall& b, bool il, cudaStream_t s) {
  const dim3 grid(b.blocks), block(128);
  if (il)
    return launch("qk_rope_backward", rope_bwd_kernel<T, T2, D, true>, grid, block, 0, s, b.a, b.dq,
                  b.dk, b.dqs, b.dks, b.gq, b.gk, b.part);
  return launch("qk_rope_backward", rope_bwd_kernel<T, T2, D, false>, grid, block, 0, s, b.a, b.dq,
                b.dk, b.dqs, b.dks, b.gq, b.gk, b.part);
}

template <typename T, typename T2>
cudaError_t dispatch_bwd(const BwdCall& b, int d, bool il, cudaStream_t s) {
  return d == 128 ? launch_bwd<T, T2, 128>(b, il, s) : launch_bwd<T, T2, 64>(b, il, s);
}

}  // namespace
}  // namespace adaspark

using namespace adaspark;

extern "C" {

int adaspark_rope_frequencies(int rot, double base, int scaling, double factor, int original_len,
                              double *freq, float *magnitude) {
  if (!freq || !magnitude || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
    return ADASPARK_EINVAL;
  if (scaling < ADASPARK_ROPE_PLAIN || scaling > ADASPARK_ROPE_YARN) return ADASPARK_EINVAL;
  if (scaling != ADASPARK_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return ADASPARK_EINVAL;
  if (scaling == ADASPARK_ROPE_NTK && rot < 4) return ADASPARK_EINVAL;
  if (scaling == ADASPARK_ROPE_YARN && original_len < 1) return ADASPARK_EINVAL;
  const int half = rot / 2;
  double b = base;
  if (scaling == ADASPARK_ROPE_NTK) b = base * std::pow(factor, rot / (rot - 2.0));
  *magnitude = 1.f;
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(b, -2.0 * i / rot);
    freq[i] = f;
    if (scaling == ADASPARK_ROPE_LINEAR) freq[i] = f / factor;
    if (scaling == ADASPARK_ROPE_YARN) {
      // r turns over the original length: f itself from 32 turns on, f / factor up
      // to one turn, and a share linear in r between them
      const double r = original_len * f / 6.283185307179586476925;
      const double keep = std::fmin(1.0, std::fmax(0.0, (r - 1.0) / 31.0));
      freq[i] = f * keep + f / factor * (1.0 - keep);
    }
  }
  if (scaling == ADASPARK_ROPE_YARN) *magnitude = (float)(0.1 * std::log(factor) + 1.0);
  return ADASPARK_OK;
}

int adaspark_qk_rope(const void* Q, int64_t q_ts, int64_t q_hs, const void* K, int64_t k_ts,
                     int64_t k_hs, int dtype, const int32_t* positions, int n_axes,
                     const int32_t* sections, const double* freq, int rot, int interleaved,
                     float magnitude, const void* w_q, const void* w_k, float eps, int n_tokens,
                     int hq, int hkv, int d, void* Q_out, int64_t qo_ts, int64_t qo_hs,
                     void* K_out, int64_t ko_ts, int64_t ko_hs, void* stream) {
  if (n_tokens < 0 || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (n_tokens == 0) return ADASPARK_OK;
  if (!Q || !K || !Q_out || !K_out) return ADASPARK_EINVAL;
  if (!rope_ok(freq, rot, d, positions, n_axes, sections, magnitude)) return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !rows_aligned(K, k_ts, k_hs, dtype) ||
      !rows_aligned(Q_out, qo_ts, qo_hs, dtype) || !rows_aligned(K_out, ko_ts, ko_hs, dtype) ||
      !aligned(w_q, 16) || !aligned(w_k, 16))
    return ADASPARK_EINVAL;
  if (!rows_distinct(n_tokens, hq, d, qo_ts, qo_hs) || !rows_distinct(n_tokens, hkv, d, ko_ts, ko_hs))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  RopeArgs a{};
  set_rope(&a, freq, rot, positions, n_axes, sections, magnitude, n_tokens);
  a.q = Q; a.k = K; a.qo = Q_out; a.ko = K_out;
  a.qs = {q_ts, q_hs}; a.ks = {k_ts, k_hs}; a.qos = {qo_ts, qo_hs}; a.kos = {ko_ts, ko_hs};
  a.wq = w_q; a.wk = w_k; a.eps = eps; a.hq = hq; a.hkv = hkv;
  return cuda_status(dispatch_rope<false>(a, dtype, d, interleaved != 0, sms,
                                          static_cast<cudaStream_t>(stream)));
}

int adaspark_qk_rope_append(const void* Q, int64_t q_ts, int64_t q_hs, const void* K, int64_t k_ts,
                            int64_t k_hs, const void* V, int64_t v_ts, int64_t v_hs, int dtype,
                            const int32_t* positions, int n_axes, const int32_t* sections,
                            const double* freq, int rot, int interleaved, float magnitude,
                            const void* w_q, const void* w_k, float eps, int n_tokens, int hq,
                            int hkv, int d, const int32_t* slots, void* k_cache, void* v_cache,
                            int64_t c_ps, int64_t c_ts, int64_t c_hs, int n_pages, int page_size,
                            void* Q_out, int64_t qo_ts, int64_t qo_hs, void* stream) {
  if (n_tokens < 0 || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (n_tokens == 0) return ADASPARK_OK;
  if (!Q || !K || !V || !Q_out || !slots) return ADASPARK_EINVAL;
  if (!rope_ok(freq, rot, d, positions, n_axes, sections, magnitude)) return ADASPARK_EINVAL;
  const CacheRows cs{c_ps, c_ts, c_hs, n_pages, page_size};
  if (!cache_ok(k_cache, v_cache, cs, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !rows_aligned(K, k_ts, k_hs, dtype) ||
      !rows_aligned(V, v_ts, v_hs, dtype) || !rows_aligned(Q_out, qo_ts, qo_hs, dtype) ||
      !aligned(w_q, 16) || !aligned(w_k, 16) || !aligned(slots, 4))
    return ADASPARK_EINVAL;
  if (!rows_distinct(n_tokens, hq, d, qo_ts, qo_hs)) return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  RopeArgs a{};
  set_rope(&a, freq, rot, positions, n_axes, sections, magnitude, n_tokens);
  a.q = Q; a.k = K; a.v = V; a.qo = Q_out;
  a.qs = {q_ts, q_hs}; a.ks = {k_ts, k_hs}; a.vs = {v_ts, v_hs}; a.qos = {qo_ts, qo_hs};
  a.wq = w_q; a.wk = w_k; a.eps = eps; a.hq = hq; a.hkv = hkv;
  a.slots = slots; a.kc = k_cache; a.vc = v_cache; a.cs = cs;
  return cuda_status(dispatch_rope<true>(a, dtype, d, interleaved != 0, sms,
                                         static_cast<cudaStream_t>(stream)));
}

int adaspark_kv_append(const void* K, int64_t k_ts, int64_t k_hs, const void* V, int64_t v_ts,
                       int64_t v_hs, int dtype, int n_tokens, int hkv, int d, const int32_t* slots,
                       void* k_cache, void* v_cache, int64_t c_ps, int64_t c_ts, int64_t c_hs,
                       int n_pages, int page_size, void* stream) {
  if (n_tokens < 0 || !head_sizes_ok(hkv, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (n_tokens == 0) return ADASPARK_OK;
  if (!K || !V || !slots) return ADASPARK_EINVAL;
  const CacheRows cs{c_ps, c_ts, c_hs, n_pages, page_size};
  if (!cache_ok(k_cache, v_cache, cs, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (!rows_aligned(K, k_ts, k_hs, dtype) || !rows_aligned(V, v_ts, v_hs, dtype) ||
      !aligned(slots, 4))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  // the append kernel with no query heads and nothing rotated
  RopeArgs a{};
  a.n = n_tokens; a.k = K; a.v = V; a.ks = {k_ts, k_hs}; a.vs = {v_ts, v_hs};
  a.hkv = hkv; a.slots = slots; a.kc = k_cache; a.vc = v_cache; a.cs = cs;
  return cuda_status(dispatch_rope<true>(a, dtype, d, false, sms,
                                         static_cast<cudaStream_t>(stream)));
}

size_t adaspark_qk_rope_backward_workspace(int n_tokens, int hq, int hkv, int d, int dtype) {
  if (n_tokens < 0 || !head_sizes_ok(hq, hkv, d, dtype)) return 0;
  return align_up((size_t)kBwdMaxBlocks * 2 * d * sizeof(float));
}

int adaspark_qk_rope_backward(const void* dQ_out, int64_t dq_ts, int64_t dq_hs, const void* dK_out,
                              int64_t dk_ts, int64_t dk_hs, int dy_dtype, const void* Q,
                              int64_t q_ts, int64_t q_hs, const void* K, int64_t k_ts,
                              int64_t k_hs, int dtype, const int32_t* positions, int n_axes,
                              const int32_t* sections, const double* freq, int rot,
                              int interleaved, float magnitude, const void* w_q, const void* w_k,
                              float eps, int n_tokens, int hq, int hkv, int d, float* dQ,
                              float* dK, float* dw_q, float* dw_k, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const bool norm = w_q || w_k;
  if (n_tokens < 0 || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype) ||
      (dy_dtype != ADASPARK_BF16 && dy_dtype != ADASPARK_FP32))
    return ADASPARK_EINVAL;
  if (!aligned(dw_q, 4) || !aligned(dw_k, 4) || (w_q && !dw_q) || (w_k && !dw_k))
    return ADASPARK_EINVAL;
  if (n_tokens == 0) {  // the weights' gradients are empty sums
    const int rc = current_device(nullptr);
    if (rc != ADASPARK_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((w_q && cudaMemsetAsync(dw_q, 0, d * sizeof(float), s) != cudaSuccess) ||
        (w_k && cudaMemsetAsync(dw_k, 0, d * sizeof(float), s) != cudaSuccess))
      return ADASPARK_ECUDA;
    return ADASPARK_OK;
  }
  if (!dQ_out || !dK_out || !dQ || !dK) return ADASPARK_EINVAL;
  if (!rope_ok(freq, rot, d, positions, n_axes, sections, magnitude)) return ADASPARK_EINVAL;
  if ((w_q && !Q) || (w_k && !K)) return ADASPARK_EINVAL;
  if (!rows_aligned(dQ_out, dq_ts, dq_hs, dy_dtype) ||
      !rows_aligned(dK_out, dk_ts, dk_hs, dy_dtype) || !aligned(dQ, 16) || !aligned(dK, 16) ||
      !aligned(w_q, 16) || !aligned(w_k, 16))
    return ADASPARK_EINVAL;
  if ((w_q && !rows_aligned(Q, q_ts, q_hs, dtype)) ||
      (w_k && !rows_aligned(K, k_ts, k_hs, dtype)))
    return ADASPARK_EINVAL;
  if (norm && (!workspace || !aligned(workspace, kAlign) ||
               workspace_bytes < adaspark_qk_rope_backward_workspace(n_tokens, hq, hkv, d, dtype)))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BwdCall b{};
  set_rope(&b.a, freq, rot, positions, n_axes, sections, magnitude, n_tokens);
  b.a.q = Q; b.a.k = K; b.a.qs = {q_ts, q_hs}; b.a.ks = {k_ts, k_hs};
  b.a.wq = w_q; b.a.wk = w_k; b.a.eps = eps; b.a.hq = hq; b.a.hkv = hkv;
  b.dq = dQ_out; b.dk = dK_out; b.dqs = {dq_ts, dq_hs}; b.dks = {dk_ts, dk_hs};
  b.gq = dQ; b.gk = dK; b.part = static_cast<float*>(workspace);
  int blocks = sms * kBwdBlocksPerSm;
  if (blocks > kBwdMaxBlocks) blocks = kBwdMaxBlocks;
  if (blocks > (n_tokens + 3) / 4) blocks = (n_tokens + 3) / 4;
  b.blocks = blocks;
  const bool il = interleaved != 0;
  using bf16 = __nv_bfloat16;
  cudaError_t e;
  if (dtype == ADASPARK_BF16)
    e = dy_dtype == ADASPARK_BF16 ? dispatch_bwd<bf16, bf16>(b, d, il, s)
                                  : dispatch_bwd<bf16, float>(b, d, il, s);
  else
    e = dy_dtype == ADASPARK_BF16 ? dispatch_bwd<float, bf16>(b, d, il, s)
                                  : dispatch_bwd<float, float>(b, d, il, s);
  if (e == cudaSuccess && norm)
    e = launch("qk_rope_dw", rope_dw_kernel, dim3(2 * d / 32), dim3(1024), 0, s, b.part, blocks, d,
               w_q ? dw_q : nullptr, w_k ? dw_k : nullptr);
  return cuda_status(e);
}

}  // extern "C"
