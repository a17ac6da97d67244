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
// exchange, and the norm's sum takes log2(d/16) shuffles. Angles are reduced to a
// turn in 64 bits (positions of 2^20 and more keep full fp32 accuracy), sines and
// cosines, norms and rotations are in 32 bits and outputs rounded once. fp32 outputs
// are off by 4.5e-8 of their size; 3.6e-8 in plain torch, whose sines are of the turn
// in 64 bits, which here would take 18559 normalised tokens 31.2 us instead of 29.9.
#include <algorithm>
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
  int32_t n, hq, hkv;
  float eps, magnitude;
};

constexpr double kInvTwoPi = 0.15915494309189533577;

// Forward: runs of 8 elements, 7 blocks on an SM for bf16 (72 registers, up to 24
// bytes spilled). One call after another, 5 to 9 blocks: 65792 tokens of 28 + 4 heads
// of 128 192, 177, 168, 179 and 187 us (at 9 up to 128 bytes are spilled); 18559
// normalised tokens of 16 + 2 heads, through the ring, 30.0, 29.4, 30.2, 31.9 and
// 39.7 us. The floors at 6.46 TB/s: 167 and 26.5 us. Blocks that end after a token, in
// the kernel's first form: 190 and 42 us.
constexpr int kRopeRun = 8;
template <typename T>
constexpr int kRopeBlocks = sizeof(T) == 2 ? 7 : 5;
// Backward: runs of 4 elements (half the values per lane beside 32 sums for the weights).
// With norms 3 blocks on an SM, rows three steps ahead: fewer warps keep the memory's order
// better. 18560 tokens of 16 + 2 normalised heads of 128, weights' gradient included, calls one
// after another: 71.8 us (floor 66); 78.6 at 6 blocks, 87.9 at 2, 74.3 two steps ahead, 71.7
// five; 161 with nothing ahead. Without norms two steps ahead (three: as at 6 blocks) and 3
// blocks for many tokens, 6 for up to two tokens a warp: 30001 tokens of 16 + 2 heads 86.4 and
// 93.0 us, 9999 of 28 + 4 53.0 and 56.7, 2999 11.9 and 11.1.
constexpr int kBwdRun = 4;
template <bool NORM>
constexpr int kBwdAhead = NORM ? 3 : 2;
template <bool NORM>
constexpr int kBwdBlocksPerSm = NORM ? 3 : 6;   // residents
constexpr int kBwdLongBlocks = 3;

// A head's lanes, each with two runs of V elements.
template <int D, int V>
struct RopeMap {
  static constexpr int kLanes = D / (2 * V);     // lanes per head
  static constexpr int kHeads = 32 / kLanes;     // heads per warp step
  static constexpr int kAngles = V / kHeads;     // angles a lane computes
  static_assert(kAngles >= 1, "");
};

// First elements of the two runs of lane `l` of a head.
template <int V>
__device__ __forceinline__ void rope_runs(int l, int rot, int* e0, int* e1) {
  const int rl = rot / (2 * V);  // rotated lanes
  if (l < rl) {
    *e0 = V * l;
    *e1 = V * l + (rot >> 1);
  } else {
    *e0 = rot + 2 * V * (l - rl);
    *e1 = *e0 + V;
  }
}

// Pair index of entry e of a rotated lane's V pairs.
template <bool IL, int V>
__device__ __forceinline__ int rope_pair(int l, int e, int rot) {
  if (!IL) return V * l + e;
  return e < V / 2 ? V / 2 * l + e : V / 2 * l + (rot >> 2) + (e - V / 2);
}

// The pairs whose angles this lane computes. The lanes of the warp that stand at
// the same place of different heads share their angles: each computes V / heads
// of them and the warp exchanges them.
template <int D, bool IL, int V>
struct RopePairs {
  using M = RopeMap<D, V>;
  double freq[M::kAngles];   // in turns per position; 0 outside the rotated part
  int64_t axis[M::kAngles];  // offset of the pair's axis of positions

  __device__ __forceinline__ RopePairs(const RopeArgs& a, int lane) {
    const int l = lane % M::kLanes, grp = lane / M::kLanes;
#pragma unroll
    for (int i = 0; i < M::kAngles; ++i) {
      freq[i] = 0.0;
      axis[i] = 0;
      if (l < a.rot / (2 * V)) {
        const int pair = rope_pair<IL, V>(l, grp * M::kAngles + i, a.rot);
        freq[i] = a.freq[pair] * kInvTwoPi;
        axis[i] = (pair < a.sec0 ? 0 : pair < a.sec01 ? 1 : 2) * a.pos_axis;
      }
    }
  }
  __device__ __forceinline__ void positions(const RopeArgs& a, int t, int (&p)[M::kAngles]) const {
#pragma unroll
    for (int i = 0; i < M::kAngles; ++i) p[i] = a.rot > 0 ? a.pos[axis[i] + t] : 0;
  }
};

// The rotation of one token for this lane's V pairs, as factors of element pairs;
// lanes outside the rotated part leave their elements alone. FULL: there are none
// (known at compile time, 18559 normalised tokens take 30.2 us instead of 31.4, 65792
// of 28 + 4 heads 168 instead of 172).
// BACK: the transpose.
template <int D, bool IL, int V, bool FULL = false>
struct RopeTurn {
  using M = RopeMap<D, V>;
  // halves: c, s, -s of elements (2i, 2i + 1); interleaved: (c, c) and (-s, s) of pair i
  F2 c[IL ? V : V / 2], s[IL ? V : V / 2], ns[IL ? 1 : V / 2];
  bool turns;

  template <bool BACK>
  __device__ __forceinline__ void set(const RopeArgs& a, const RopePairs<D, IL, V>& pairs,
                                      const int (&p)[M::kAngles], int lane) {
    const int l = lane % M::kLanes;
    float mc[M::kAngles], ms[M::kAngles];
#pragma unroll
    for (int i = 0; i < M::kAngles; ++i) {
      const double turn = (double)p[i] * pairs.freq[i];
      float sn, cn;
      sincospif(2.f * (float)(turn - rint(turn)), &sn, &cn);
      mc[i] = cn * a.magnitude;
      ms[i] = (BACK ? -sn : sn) * a.magnitude;
    }
    float ce[V], se[V];
    turns = l < a.rot / (2 * V);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int src = (e / M::kAngles) * M::kLanes + l;
      ce[e] = __shfl_sync(0xffffffffu, mc[e % M::kAngles], src);
      se[e] = __shfl_sync(0xffffffffu, ms[e % M::kAngles], src);
    }
    if (IL) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        c[e % (IL ? V : V / 2)] = f2(ce[e], ce[e]);
        s[e % (IL ? V : V / 2)] = f2(-se[e], se[e]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        c[i] = f2(ce[2 * i], ce[2 * i + 1]);
        s[i] = f2(se[2 * i], se[2 * i + 1]);
        ns[i % (IL ? 1 : V / 2)] = f2(-se[2 * i], -se[2 * i + 1]);
      }
    }
  }

  // Rotates a lane's two runs in place.
  __device__ __forceinline__ void turn(F2 (&u)[V / 2], F2 (&v)[V / 2]) const {
    if (!FULL && !turns) return;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (IL) {
        const float2 x = unpack(u[i]), y = unpack(v[i]);
        u[i] = fma2(f2(x.y, x.x), s[i], mul2(u[i], c[i]));
        v[i] = fma2(f2(y.y, y.x), s[(V / 2 + i) % (IL ? V : V / 2)],
                    mul2(v[i], c[(V / 2 + i) % (IL ? V : V / 2)]));
      } else {
        const F2 x = u[i], y = v[i];
        u[i] = fma2(y, ns[i % (IL ? 1 : V / 2)], mul2(x, c[i]));
        v[i] = fma2(x, s[i], mul2(y, c[i]));
      }
    }
  }
};

template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Norm weights of queries and keys in fp32, ones where there is none.
template <typename T, int D>
__device__ __forceinline__ void rope_weights(const RopeArgs& a, float (&w)[2][D]) {
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
    const T* p = static_cast<const T*>(i < D ? a.wq : a.wk);
    w[i / D][i % D] = p ? to_f32(p[i % D]) : 1.f;
  }
  __syncthreads();
}
template <int V>
__device__ __forceinline__ void load_f2(const float* p, F2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 x = reinterpret_cast<const float4*>(p)[i];
    v[2 * i] = f2(x.x, x.y);
    v[2 * i + 1] = f2(x.z, x.w);
  }
}
// Sum of the squares of a head's elements.
template <int V, int LANES>
__device__ __forceinline__ float head_squares(const F2 (&u)[V / 2], const F2 (&v)[V / 2]) {
  F2 ss = mul2(u[0], u[0]);
#pragma unroll
  for (int i = 1; i < V / 2; ++i) ss = fma2(u[i], u[i], ss);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) ss = fma2(v[i], v[i], ss);
  const float2 two = unpack(ss);
  return head_sum<LANES>(two.x + two.y);
}

// A lane's two runs of a row, as they lie in memory; `gap`: elements between them.
template <typename T, int V>
struct RopeRow {
  Raw<T, V> u, v;
  __device__ __forceinline__ void load(const T* p, int gap) {
    u.load(p);
    v.load(p + gap);
  }
  __device__ __forceinline__ void store(T* p, int gap) const {
    u.store(p);
    v.store(p + gap);
  }
};

// Norm and rotation of a row.
template <typename T, int D, bool IL, bool NORM, int V, bool FULL>
__device__ __forceinline__ void rope_head(RopeRow<T, V>& row,
                                          const RopeTurn<D, IL, V, FULL>& rotation, const float* w,
                                          bool has_w, int e0, int gap, float eps) {
  F2 u[V / 2], v[V / 2];
  row.u.get(u);
  row.v.get(v);
  if constexpr (NORM) {
    const float sum = head_squares<V, RopeMap<D, V>::kLanes>(u, v);
    const float r = has_w ? rsqrtf(fmaf(sum, 1.f / D, eps)) : 1.f;
    const F2 rr = f2(r, r);
    F2 f[V / 2];
    load_f2<V>(w + e0, f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) u[i] = mul2(mul2(u[i], rr), f[i]);
    load_f2<V>(w + e0 + gap, f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = mul2(mul2(v[i], rr), f[i]);
  }
  rotation.turn(u, v);
  row.u.set(u);
  row.v.set(v);
}

template <typename T, bool CACHE>
__device__ __forceinline__ int64_t rope_slot(const RopeArgs& a, int t) {
  if (!CACHE) return -1;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.cs.n_pages * a.cs.page_size) return -1;
  const int page = slot / a.cs.page_size;
  return page * a.cs.ps + (slot - page * a.cs.page_size) * a.cs.ts;
}

constexpr int kRopeAhead = 2;
// Rows on their way, in the order of the walk: queries, keys, (with a cache) values,
// then the warp's next token. RING: lane-private slots in shared memory, filled by
// cp.async kRopeAhead steps ahead; else registers, one step ahead.
template <typename T, int D, int V, bool CACHE, bool RING>
struct RopeRing {
  using M = RopeMap<D, V>;
  static constexpr int kPieces = V * (int)sizeof(T) / 16;  // 16-byte pieces of a run
  static constexpr int kStep = 32 * 16 * 2 * kPieces, kSlots = kRopeAhead + 1;
  static constexpr int kWarp = RING ? kSlots * kStep : 0;
  static constexpr int kAhead = RING ? kRopeAhead : 1;

  const RopeArgs& a;
  const T *q0, *k0, *v0, *p;  // of this lane's first run
  uint8_t* slots;             // this lane's part of the warp's ring
  int gap, grp, stride, q_steps, k_steps;
  int t, h, left, in, out, part;
  RopeRow<T, V> next;

  __device__ __forceinline__ void start(int token) {
    t = token;
    h = grp;
    left = q_steps;
    in = out = part = 0;
    p = q0 + t * a.qs.ts;
  }
  // Copies the walk's step into the next slot and moves on; one commit group.
  __device__ __forceinline__ void fetch() {
    if (t < a.n) {
      if (h < (part ? a.hkv : a.hq)) {
        if (RING) {
          uint8_t* s = slots + in * kStep;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            cp_async<16>(s + 512 * i, p + i * (16 / (int)sizeof(T)));
            cp_async<16>(s + 512 * (kPieces + i), p + gap + i * (16 / (int)sizeof(T)));
          }
        } else {
          next.load(p, gap);
        }
      }
      h += M::kHeads;
      if (--left > 0) {
        p += M::kHeads * (part == 0 ? a.qs.hs : part == 1 ? a.ks.hs : a.vs.hs);
      } else {
        h = grp;
        part = part == (CACHE ? 2 : 1) ? 0 : part + 1;
        left = part ? k_steps : q_steps;
        if (part == 0) t += stride;
        p = part == 0 ? q0 + t * a.qs.ts : part == 1 ? k0 + t * a.ks.ts : v0 + t * a.vs.ts;
      }
    }
    if (RING) {
      cp_async_commit();
      in = in + 1 == kSlots ? 0 : in + 1;
    }
  }
  // The next row of the walk; a step is copied into the slot that the one before has used up.
  __device__ __forceinline__ RopeRow<T, V> take() {
    RopeRow<T, V> r = next;
    fetch();
    if (!RING) return r;
    cp_async_wait<kRopeAhead>();
    const uint8_t* s = slots + out * kStep;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(s + 512 * i);
      const uint4 y = *reinterpret_cast<const uint4*>(s + 512 * (kPieces + i));
      r.u.w[4 * i] = x.x; r.u.w[4 * i + 1] = x.y; r.u.w[4 * i + 2] = x.z; r.u.w[4 * i + 3] = x.w;
      r.v.w[4 * i] = y.x; r.v.w[4 * i + 1] = y.y; r.v.w[4 * i + 2] = y.z; r.v.w[4 * i + 3] = y.w;
    }
    out = out + 1 == kSlots ? 0 : out + 1;
    return r;
  }
};

// Many tokens: warps walk tokens; queries, then keys, then (with a cache) values,
// which are copied.
template <typename T, int D, bool IL, bool CACHE, bool NORM, bool FULL, bool RING>
__global__ void __launch_bounds__(128, kRopeBlocks<T>) rope_walk_kernel(const RopeArgs a) {
  constexpr int V = kRopeRun;
  using M = RopeMap<D, V>;
  using Ring = RopeRing<T, D, V, CACHE, RING>;
  __shared__ __align__(16) float weights[2][NORM ? D : 1];
  extern __shared__ __align__(16) uint8_t rings[];
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / M::kLanes;
  const int stride = gridDim.x * 4;
  int e0, e1;
  rope_runs<V>(lane % M::kLanes, a.rot, &e0, &e1);
  const int gap = e1 - e0;
  const int q_steps = (a.hq + M::kHeads - 1) / M::kHeads;
  const int k_steps = (a.hkv + M::kHeads - 1) / M::kHeads;
  int t = blockIdx.x * 4 + warp;
  Ring ring{a,
            static_cast<const T*>(a.q) + grp * a.qs.hs + e0,
            static_cast<const T*>(a.k) + grp * a.ks.hs + e0,
            CACHE ? static_cast<const T*>(a.v) + grp * a.vs.hs + e0 : nullptr,
            nullptr,
            rings + warp * Ring::kWarp + lane * 16,
            gap,
            grp,
            stride,
            q_steps,
            k_steps};
  ring.start(t);
#pragma unroll
  for (int i = 0; i < Ring::kAhead; ++i) ring.fetch();
  const RopePairs<D, IL, V> pairs(a, lane);
  int pos[M::kAngles] = {};
  if (t < a.n) pairs.positions(a, t, pos);
  if constexpr (NORM) rope_weights<T, D>(a, weights);
  RopeTurn<D, IL, V, FULL> rotation;
  for (; t < a.n; t += stride) {
    const int64_t slot = rope_slot<T, CACHE>(a, t);
    rotation.template set<false>(a, pairs, pos, lane);
    if (t + stride < a.n) pairs.positions(a, t + stride, pos);
    T* o = static_cast<T*>(a.qo) + t * a.qos.ts + grp * a.qos.hs + e0;
    for (int h = grp, st = 0; st < q_steps; ++st, h += M::kHeads) {
      RopeRow<T, V> row = ring.take();
      rope_head<T, D, IL, NORM>(row, rotation, weights[0], a.wq != nullptr, e0, gap, a.eps);
      if (h < a.hq) row.store(o, gap);
      o += M::kHeads * a.qos.hs;
    }
    const int64_t ostep = M::kHeads * (CACHE ? a.cs.hs : a.kos.hs);
    o = CACHE ? static_cast<T*>(a.kc) + (slot + grp * a.cs.hs + e0)
              : static_cast<T*>(a.ko) + t * a.kos.ts + grp * a.kos.hs + e0;
    for (int h = grp, st = 0; st < k_steps; ++st, h += M::kHeads) {
      RopeRow<T, V> row = ring.take();
      rope_head<T, D, IL, NORM>(row, rotation, weights[NORM ? 1 : 0], a.wk != nullptr, e0, gap,
                                a.eps);
      if (h < a.hkv && (!CACHE || slot >= 0)) row.store(o, gap);
      o += ostep;
    }
    if (CACHE) {
      o = static_cast<T*>(a.vc) + (slot + grp * a.cs.hs + e0);
      for (int h = grp, st = 0; st < k_steps; ++st, h += M::kHeads) {
        const RopeRow<T, V> row = ring.take();
        if (h < a.hkv && slot >= 0) row.store(o, gap);
        o += ostep;
      }
    }
  }
  if (RING) cp_async_wait<0>();
}

// Few tokens: a warp per step of a token's heads.
// Latency-bound: one token of 28 + 4 normalised heads, one call after another, 2.1 us,
// 200 tokens of 16 + 2 heads 1.8 us.
template <typename T, int D, bool IL, bool CACHE, bool NORM>
__global__ void __launch_bounds__(128) rope_step_kernel(const RopeArgs a) {
  constexpr int V = kRopeRun;
  using M = RopeMap<D, V>;
  __shared__ __align__(16) float weights[2][NORM ? D : 1];
  dependency_wait();
  const int lane = threadIdx.x & 31, grp = lane / M::kLanes;
  const int q_steps = (a.hq + M::kHeads - 1) / M::kHeads;
  const int k_steps = (a.hkv + M::kHeads - 1) / M::kHeads;
  const int steps = q_steps + k_steps * (CACHE ? 2 : 1);
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5), t = item / steps;
  int st = item - t * steps, part = 0;  // 0 queries, 1 keys, 2 values
  if (st >= q_steps) {
    st -= q_steps;
    part = 1;
    if (CACHE && st >= k_steps) {
      st -= k_steps;
      part = 2;
    }
  }
  const int h = st * M::kHeads + grp;
  const bool mine = t < a.n && h < (part ? a.hkv : a.hq);
  int e0, e1;
  rope_runs<V>(lane % M::kLanes, a.rot, &e0, &e1);
  const int gap = e1 - e0;
  RopeRow<T, V> row{};
  if (mine) {
    const HeadRows s = part == 0 ? a.qs : part == 1 ? a.ks : a.vs;
    row.load(static_cast<const T*>(part == 0 ? a.q : part == 1 ? a.k : a.v) + t * s.ts + h * s.hs +
                 e0, gap);
  }
  if constexpr (NORM) rope_weights<T, D>(a, weights);
  if (t >= a.n) return;
  const int64_t slot = part ? rope_slot<T, CACHE>(a, t) : -1;
  if (part < 2) {
    const RopePairs<D, IL, V> pairs(a, lane);
    int pos[M::kAngles];
    pairs.positions(a, t, pos);
    RopeTurn<D, IL, V> rotation;
    rotation.template set<false>(a, pairs, pos, lane);
    rope_head<T, D, IL, NORM>(row, rotation, weights[NORM ? part : 0],
                                 (part ? a.wk : a.wq) != nullptr, e0, gap, a.eps);
  }
  if (!mine) return;
  if (part == 0)
    row.store(static_cast<T*>(a.qo) + t * a.qos.ts + h * a.qos.hs + e0, gap);
  else if (!CACHE)
    row.store(static_cast<T*>(a.ko) + t * a.kos.ts + h * a.kos.hs + e0, gap);
  else if (slot >= 0)
    row.store(static_cast<T*>(part == 1 ? a.kc : a.vc) + slot + h * a.cs.hs + e0, gap);
}

// Keys and values as they are into the cache, 16 bytes at a time, kCopyAhead of them in
// flight per thread. HBM-bound: 65792 tokens of 4 heads of 128, bf16, one call after another
// 44.1 us (floor 41.7), 18559 of 2 heads 8.9 (5.9), 64 tokens 2.6; with two in flight 46.1, 8.8
// and 1.9, with eight 47.3, 9.3 and 4.0; a warp per token's heads 48.7 and 14.1.
constexpr int kCopyThreads = 128, kCopyAhead = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const RopeArgs a) {
  constexpr int kPer = 16 / (int)sizeof(T), kPieces = D / kPer;  // pieces of a head
  dependency_wait();
  const int row = a.hkv * kPieces, both = 2 * row;
  // the block's first piece: of token t0, r0 pieces into its keys and values
  const int64_t base = (int64_t)blockIdx.x * (kCopyThreads * kCopyAhead);
  const int t0 = (int)(base / both), r0 = (int)(base - (int64_t)t0 * both);
  uint4 v[kCopyAhead];
  T* to[kCopyAhead];
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i) {
    const int r = r0 + i * kCopyThreads + (int)threadIdx.x, dt = r / both, t = t0 + dt;
    to[i] = nullptr;
    if (t >= a.n) continue;
    const int64_t slot = rope_slot<T, true>(a, t);
    if (slot < 0) continue;
    int p = r - dt * both;
    const bool value = p >= row;
    if (value) p -= row;
    const int h = p / kPieces, e = p % kPieces * kPer;
    const HeadRows s = value ? a.vs : a.ks;
    v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(value ? a.v : a.k) + t * s.ts +
                                           h * s.hs + e);
    to[i] = static_cast<T*>(value ? a.vc : a.kc) + slot + h * a.cs.hs + e;
  }
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i)
    if (to[i]) *reinterpret_cast<uint4*>(to[i]) = v[i];
}

// Rows of the backward pass on their way: lane-private slots in shared memory, a
// ring of kAhead + 1 steps filled by cp.async (registers would hold one step
// ahead). The walk: queries, then keys, then the warp's next token.
template <typename T, typename T2, int D, int V, bool NORM>
struct BwdRing {
  using M = RopeMap<D, V>;
  static constexpr int kDy = V * (int)sizeof(T2), kX = V * (int)sizeof(T);  // bytes of a run
  static constexpr int kStep = 32 * 2 * (kDy + (NORM ? kX : 0));
  static constexpr int kAhead = kBwdAhead<NORM>, kSlots = kAhead + 1;
  static constexpr int kWarp = kSlots * kStep;

  const RopeArgs& a;
  const T2 *dq0, *dk0, *dy;   // of this lane's first run
  const T *q0, *k0, *x;
  HeadRows dqs, dks;
  uint8_t* slots;             // this lane's part of the warp's ring
  int gap, grp, stride, q_steps, k_steps;
  int t, h, left, slot;
  bool keys;

  __device__ __forceinline__ void start(int token) {
    t = token;
    keys = false;
    h = grp;
    left = q_steps;
    slot = 0;
    dy = dq0 + t * dqs.ts;
    x = q0 + t * a.qs.ts;
  }
  // Copies the walk's step into the next slot and moves on; one commit group.
  __device__ __forceinline__ void fetch() {
    if (t < a.n) {
      if (h < (keys ? a.hkv : a.hq)) {
        uint8_t* s = slots + slot * kStep;
        cp_async<kDy>(s, dy);
        cp_async<kDy>(s + 32 * kDy, dy + gap);
        if (NORM && (keys ? a.wk : a.wq)) {
          // rows start on 16 bytes, a lane's runs on 8 or 16 of them
          uint8_t* sx = slot_x(slot);
          cp_async<kX>(sx, x);
          cp_async<kX>(sx + 32 * kX, x + gap);
        }
      }
      h += M::kHeads;
      if (--left > 0) {
        dy += M::kHeads * (keys ? dks.hs : dqs.hs);
        x += M::kHeads * (keys ? a.ks.hs : a.qs.hs);
      } else {
        h = grp;
        keys = !keys;
        left = keys ? k_steps : q_steps;
        if (!keys) t += stride;
        dy = keys ? dk0 + t * dks.ts : dq0 + t * dqs.ts;
        x = keys ? k0 + t * a.ks.ts : q0 + t * a.qs.ts;
      }
    }
    cp_async_commit();
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  __device__ __forceinline__ uint8_t* slot_x(int i) const {
    const int lane = threadIdx.x & 31;
    return slots - lane * kDy + i * kStep + 64 * kDy + lane * kX;
  }
  __device__ __forceinline__ void row(int i, RopeRow<T2, V>& dy_row, RopeRow<T, V>& x_row) const {
    const uint8_t* s = slots + i * kStep;
    dy_row.u.load(reinterpret_cast<const T2*>(s));
    dy_row.v.load(reinterpret_cast<const T2*>(s + 32 * kDy));
    if (NORM) {
      const uint8_t* sx = slot_x(i);
      x_row.u.load(reinterpret_cast<const T*>(sx));
      x_row.v.load(reinterpret_cast<const T*>(sx + 32 * kX));
    }
  }
};

// Backward: warps walk tokens with a fixed stride, so the partial sums of the
// weights' gradients have a fixed order; each block writes one row of them.
// dy in T2, x in T, dx in fp32.
template <typename T, typename T2, int D, bool IL, bool NORM>
__global__ void __launch_bounds__(128, kBwdBlocksPerSm<NORM>)
    rope_bwd_kernel(const RopeArgs a, const void* dq, const void* dk, HeadRows dqs, HeadRows dks,
                    float* gq, float* gk, float* part) {
  constexpr int V = kBwdRun;
  using M = RopeMap<D, V>;
  using Ring = BwdRing<T, T2, D, V, NORM>;
  __shared__ __align__(16) float weights[2][NORM ? D : 1];
  __shared__ __align__(16) uint8_t rings[4 * Ring::kWarp];
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / M::kLanes;
  int e0, e1;
  rope_runs<V>(lane % M::kLanes, a.rot, &e0, &e1);
  const int gap = e1 - e0, stride = gridDim.x * 4;
  const int q_steps = (a.hq + M::kHeads - 1) / M::kHeads;
  const int k_steps = (a.hkv + M::kHeads - 1) / M::kHeads;
  const bool has_q = NORM && a.wq, has_k = NORM && a.wk;
  F2 dwq[V] = {}, dwk[V] = {};
  int t = blockIdx.x * 4 + warp;
  Ring ring{a,
            static_cast<const T2*>(dq) + grp * dqs.hs + e0,
            static_cast<const T2*>(dk) + grp * dks.hs + e0,
            nullptr,
            static_cast<const T*>(a.q) + grp * a.qs.hs + e0,
            static_cast<const T*>(a.k) + grp * a.ks.hs + e0,
            nullptr,
            dqs,
            dks,
            rings + warp * Ring::kWarp + lane * Ring::kDy,
            gap,
            grp,
            stride,
            q_steps,
            k_steps};
  ring.start(t);
#pragma unroll
  for (int i = 0; i < Ring::kAhead; ++i) ring.fetch();
  const RopePairs<D, IL, V> pairs(a, lane);
  int pos[M::kAngles] = {};
  if (t < a.n) pairs.positions(a, t, pos);
  if constexpr (NORM) rope_weights<T, D>(a, weights);
  RopeTurn<D, IL, V> rotation;
  int slot = 0;

  // dx of the next row from dy and x; its weights' gradient onto dw.
  auto head = [&](const float* w, bool has_w, F2 (&dw)[V], float* o, bool mine) {
    ring.fetch();  // into the slot that the step before has used up
    cp_async_wait<Ring::kAhead>();
    RopeRow<T2, V> dy;
    RopeRow<T, V> xr;
    ring.row(slot, dy, xr);
    slot = slot + 1 == Ring::kSlots ? 0 : slot + 1;
    F2 u[V / 2], v[V / 2];
    dy.u.get(u);
    dy.v.get(v);
    rotation.turn(u, v);
    if (NORM && has_w) {
      F2 x[V / 2], y[V / 2], f[V / 2];
      xr.u.get(x);
      xr.v.get(y);
      const float r = rsqrtf(fmaf(head_squares<V, M::kLanes>(x, y), 1.f / D, a.eps));
      const F2 rr = f2(r, r);
      F2 dd = f2(0.f, 0.f);
      load_f2<V>(w + e0, f);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x[i] = mul2(x[i], rr);
        if (mine) dw[i] = fma2(u[i], x[i], dw[i]);
        u[i] = mul2(u[i], f[i]);
        dd = fma2(u[i], x[i], dd);
      }
      load_f2<V>(w + e1, f);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        y[i] = mul2(y[i], rr);
        if (mine) dw[V / 2 + i] = fma2(v[i], y[i], dw[V / 2 + i]);
        v[i] = mul2(v[i], f[i]);
        dd = fma2(v[i], y[i], dd);
      }
      const float2 d2 = unpack(dd);
      const float dot = head_sum<M::kLanes>(d2.x + d2.y) * (-1.f / D);
      const F2 nd = f2(dot, dot);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        u[i] = mul2(rr, fma2(x[i], nd, u[i]));
        v[i] = mul2(rr, fma2(y[i], nd, v[i]));
      }
    }
    if (mine) {
      RopeRow<float, V> out;
      out.u.set(u);
      out.v.set(v);
      out.store(o, gap);
    }
  };
  for (; t < a.n; t += stride) {
    rotation.template set<true>(a, pairs, pos, lane);
    if (t + stride < a.n) pairs.positions(a, t + stride, pos);
    float* o = gq + ((int64_t)t * a.hq + grp) * D + e0;
    for (int h = grp, st = 0; st < q_steps; ++st, h += M::kHeads) {
      head(weights[0], has_q, dwq, o, h < a.hq);
      o += M::kHeads * D;
    }
    o = gk + ((int64_t)t * a.hkv + grp) * D + e0;
    for (int h = grp, st = 0; st < k_steps; ++st, h += M::kHeads) {
      head(weights[NORM ? 1 : 0], has_k, dwk, o, h < a.hkv);
      o += M::kHeads * D;
    }
  }
  cp_async_wait<0>();
  if constexpr (NORM) {
    // the rings are used up: their memory takes the heads' sums
    static_assert(sizeof(rings) >= sizeof(float) * 4 * M::kHeads * 2 * D, "");
    float(*sum)[2][D] = reinterpret_cast<float(*)[2][D]>(rings);
    __syncthreads();
    float(*mine)[D] = sum[warp * M::kHeads + grp];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i < V / 2 ? e0 + 2 * i : e1 + 2 * i - V;
      const float2 a2 = unpack(dwq[i]), b2 = unpack(dwk[i]);
      mine[0][e] = a2.x;
      mine[0][e + 1] = a2.y;
      mine[1][e] = b2.x;
      mine[1][e + 1] = b2.y;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += 128) {
      float acc = 0.f;
#pragma unroll
      for (int g = 0; g < 4 * M::kHeads; ++g) acc += sum[g][i / D][i % D];
      part[(int64_t)blockIdx.x * 2 * D + i] = acc;
    }
  }
}

// Sums the blocks' rows, 8 columns per block: column c of rows y, y + 128, ..., then
// over y in halves. Latency-bound: 2.6 us for 444 rows of 256.
__global__ void __launch_bounds__(1024)
    rope_dw_kernel(WsHeader* hdr, const float* part, int rows, int d, float* dwq, float* dwk) {
  __shared__ float sum[128][9];
  dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) hdr->status = hdr->detail = hdr->n_block_status = 0;
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + x;
  float acc = 0.f;
#pragma unroll 6
  for (int r = y; r < rows; r += 128) acc += part[(int64_t)r * 2 * d + col];
  sum[y][x] = acc;
  __syncthreads();
#pragma unroll
  for (int half = 64; half > 0; half >>= 1) {
    if (y < half) sum[y][x] += sum[y + half][x];
    __syncthreads();
  }
  if (y == 0) {
    float* o = col < d ? dwq : dwk;
    if (o) o[col % d] = sum[0][x];
  }
}

bool qk_rope_args_ok(const double* freq, int rot, int d, const int32_t* positions, int n_axes,
                     const int32_t* sections, float magnitude, const void* w_q, const void* w_k,
                     float eps) {
  if (!(eps >= 0.f) || !aligned(w_q, 16) || !aligned(w_k, 16)) return false;
  if (rot < 0 || rot > d || rot % 16 != 0 || !std::isfinite(magnitude)) return false;
  if (rot == 0) return true;  // positions, axes, sections and freq are not looked at
  if (!freq || !positions || !aligned(freq, 8) || !aligned(positions, 4)) return false;
  if (n_axes == 1) return true;
  if (n_axes != 3 || !sections) return false;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (sections[i] < 0) return false;
    sum += sections[i];
  }
  return sum == rot / 2;
}

namespace {

constexpr int kBwdMaxParts = 148 * kBwdBlocksPerSm<true>;  // blocks with sums for the weights

void set_rope(RopeArgs* a, const double* freq, int rot, const int32_t* positions, int n_axes,
              const int32_t* sections, float magnitude, int n) {
  const bool axes = rot > 0 && n_axes == 3;
  a->freq = freq;
  a->rot = rot;
  a->pos = positions;
  a->pos_axis = axes ? n : 0;
  a->sec0 = axes ? sections[0] : rot / 2;
  a->sec01 = axes ? sections[0] + sections[1] : rot / 2;
  a->magnitude = magnitude;
  a->n = n;
}

// bf16 rows up to this size are read through the ring, two steps ahead. Calls one after
// another, ring and registers: 2999 tokens of 16 + 2 heads of 128 5.8 and 7.0 us, 18559 (85
// MB) normalised 29.9 and 33.4; 9999 of 28 + 4 28.3 and 30.0, 14999 (123 MB) 43.3 and 41.9,
// 65792 182 and 167: there the reads that run ahead disturb the memory's order, which warps in
// step keep. Three steps ahead cost 0.3 us of 30, one 0.5. fp32, 4999 tokens: 25 and 18 us.
constexpr int64_t kRopeRingBytes = 100 << 20;

template <typename T, int D, bool CACHE, bool NORM, bool RING>
cudaError_t launch_walk(const RopeArgs& a, bool il, const char* name, dim3 grid, cudaStream_t s) {
  auto* kernel = a.rot == D ? (il ? rope_walk_kernel<T, D, true, CACHE, NORM, true, RING>
                                  : rope_walk_kernel<T, D, false, CACHE, NORM, true, RING>)
                            : (il ? rope_walk_kernel<T, D, true, CACHE, NORM, false, RING>
                                  : rope_walk_kernel<T, D, false, CACHE, NORM, false, RING>);
  constexpr int smem = 4 * RopeRing<T, D, kRopeRun, CACHE, RING>::kWarp;
  if (smem && allow_smem(kernel, smem) != ADASPARK_OK) return cudaErrorUnknown;
  return launch_after(name, kernel, grid, dim3(128), smem, s, 1, a);
}

template <typename T, int D, bool CACHE, bool NORM>
cudaError_t launch_rope(const RopeArgs& a, bool il, int sms, cudaStream_t s) {
  constexpr int H = RopeMap<D, kRopeRun>::kHeads;
  const int64_t q_steps = (a.hq + H - 1) / H, k_steps = (a.hkv + H - 1) / H;
  const int64_t steps = q_steps + k_steps * (CACHE ? 2 : 1), n = a.n;
  // A warp per step for few tokens, warps that walk whole tokens for many, from a share of the
  // resident warps that fits what was measured with norms (a warp per step, walking): bf16
  // append of 28 + 4 heads, 1200 tokens 7.6 and 7.7 us, 1600 9.7 and 8.1; rope of 4 + 1 heads,
  // 2400 tokens 4.0 and 4.1, 3600 5.5 and 4.8; fp32 rope of 28 + 4, 1200 tokens 10.6 and 11.0,
  // 1600 12.9 and 12.8.
  const int64_t warps = (int64_t)sms * kRopeBlocks<T> * 4;
  const bool walk = n > (sizeof(T) == 2 ? 0.22 + 0.65 / steps : 0.54) * warps;
  const char* name = CACHE ? "qk_rope_append" : "qk_rope";
  const dim3 block(128);
  if (walk) {
    const int64_t want = (n + 3) / 4, most = (int64_t)sms * kRopeBlocks<T>;
    const dim3 grid((unsigned)(want < most ? want : most));
    const int64_t bytes = n * (a.hq + a.hkv * (CACHE ? 2 : 1)) * D * (int64_t)sizeof(T);
    if constexpr (sizeof(T) == 2)
      if (bytes <= kRopeRingBytes) return launch_walk<T, D, CACHE, NORM, true>(a, il, name, grid, s);
    return launch_walk<T, D, CACHE, NORM, false>(a, il, name, grid, s);
  }
  const dim3 grid((unsigned)((n * steps + 3) / 4));
  return il ? launch_after(name, rope_step_kernel<T, D, true, CACHE, NORM>, grid, block, 0, s, 1, a)
            : launch_after(name, rope_step_kernel<T, D, false, CACHE, NORM>, grid, block, 0, s, 1, a);
}

template <typename T, int D, bool CACHE>
cudaError_t launch_rope(const RopeArgs& a, bool il, int sms, cudaStream_t s) {
  return a.wq || a.wk ? launch_rope<T, D, CACHE, true>(a, il, sms, s)
                      : launch_rope<T, D, CACHE, false>(a, il, sms, s);
}

template <bool CACHE>
cudaError_t dispatch_rope(const RopeArgs& a, int dtype, int d, bool il, int sms, cudaStream_t s) {
  if (dtype == ADASPARK_BF16)
    return d == 128 ? launch_rope<__nv_bfloat16, 128, CACHE>(a, il, sms, s)
                    : launch_rope<__nv_bfloat16, 64, CACHE>(a, il, sms, s);
  return d == 128 ? launch_rope<float, 128, CACHE>(a, il, sms, s)
                  : launch_rope<float, 64, CACHE>(a, il, sms, s);
}

template <typename T>
cudaError_t launch_copy(const RopeArgs& a, int d, cudaStream_t s) {
  const int64_t pieces = (int64_t)a.n * 2 * a.hkv * (d * (int)sizeof(T) / 16);
  const int64_t blocks = (pieces - 1) / (kCopyThreads * kCopyAhead) + 1;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_after("kv_append", d == 128 ? kv_copy_kernel<T, 128> : kv_copy_kernel<T, 64>,
                      dim3((unsigned)blocks), dim3(kCopyThreads), 0, s, 1, a);
}

struct BwdCall {
  RopeArgs a;
  const void *dq, *dk;
  HeadRows dqs, dks;
  float *gq, *gk, *part;
  int blocks;
};

template <typename T, typename T2, int D, bool NORM>
cudaError_t launch_bwd(const BwdCall& b, bool il, cudaStream_t s) {
  auto* kernel = il ? rope_bwd_kernel<T, T2, D, true, NORM> : rope_bwd_kernel<T, T2, D, false, NORM>;
  return launch_after("qk_rope_backward", kernel, dim3(b.blocks), dim3(128), 0, s, 1, b.a, b.dq,
                      b.dk, b.dqs, b.dks, b.gq, b.gk, b.part);
}

template <typename T, typename T2, int D>
cudaError_t launch_bwd(const BwdCall& b, bool il, cudaStream_t s) {
  return b.a.wq || b.a.wk ? launch_bwd<T, T2, D, true>(b, il, s)
                          : launch_bwd<T, T2, D, false>(b, il, s);
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
  if (n_tokens < 0 || n_tokens > (1 << 30) || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype))
    return ADASPARK_EINVAL;
  if (n_tokens == 0) return ADASPARK_OK;
  if (!Q || !K || !Q_out || !K_out) return ADASPARK_EINVAL;
  if (!qk_rope_args_ok(freq, rot, d, positions, n_axes, sections, magnitude, w_q, w_k, eps))
    return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !rows_aligned(K, k_ts, k_hs, dtype) ||
      !rows_aligned(Q_out, qo_ts, qo_hs, dtype) || !rows_aligned(K_out, ko_ts, ko_hs, dtype))
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
  if (n_tokens < 0 || n_tokens > (1 << 30) || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype))
    return ADASPARK_EINVAL;
  if (n_tokens == 0) return ADASPARK_OK;
  if (!Q || !K || !V || !Q_out || !slots) return ADASPARK_EINVAL;
  if (!qk_rope_args_ok(freq, rot, d, positions, n_axes, sections, magnitude, w_q, w_k, eps))
    return ADASPARK_EINVAL;
  const CacheRows cs{c_ps, c_ts, c_hs, n_pages, page_size};
  if (!cache_ok(k_cache, v_cache, cs, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !rows_aligned(K, k_ts, k_hs, dtype) ||
      !rows_aligned(V, v_ts, v_hs, dtype) || !rows_aligned(Q_out, qo_ts, qo_hs, dtype) ||
      !aligned(slots, 4))
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
  if (n_tokens < 0 || n_tokens > (1 << 30) || !head_sizes_ok(hkv, hkv, d, dtype))
    return ADASPARK_EINVAL;
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
  RopeArgs a{};
  a.n = n_tokens; a.k = K; a.v = V; a.ks = {k_ts, k_hs}; a.vs = {v_ts, v_hs};
  a.hkv = hkv; a.slots = slots; a.kc = k_cache; a.vc = v_cache; a.cs = cs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(dtype == ADASPARK_BF16 ? launch_copy<__nv_bfloat16>(a, d, s)
                                            : launch_copy<float>(a, d, s));
}

size_t adaspark_qk_rope_backward_workspace(int n_tokens, int hq, int hkv, int d, int dtype) {
  if (n_tokens < 0 || n_tokens > (1 << 30) || !head_sizes_ok(hq, hkv, d, dtype)) return 0;
  return align_up(sizeof(WsHeader)) + align_up((size_t)kBwdMaxParts * 2 * d * sizeof(float));
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
  if (n_tokens < 0 || n_tokens > (1 << 30) || !(eps >= 0.f) || !head_sizes_ok(hq, hkv, d, dtype) ||
      (dy_dtype != ADASPARK_BF16 && dy_dtype != ADASPARK_FP32))
    return ADASPARK_EINVAL;
  if (!aligned(dw_q, 4) || !aligned(dw_k, 4) || (w_q && !dw_q) || (w_k && !dw_k))
    return ADASPARK_EINVAL;
  if (n_tokens == 0) {  // the weights' gradients are empty sums
    const int rc = current_device(nullptr);
    if (rc != ADASPARK_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((norm && workspace && aligned(workspace, kAlign) && workspace_bytes >= sizeof(WsHeader) &&
         cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) ||
        (w_q && cudaMemsetAsync(dw_q, 0, d * sizeof(float), s) != cudaSuccess) ||
        (w_k && cudaMemsetAsync(dw_k, 0, d * sizeof(float), s) != cudaSuccess))
      return ADASPARK_ECUDA;
    return ADASPARK_OK;
  }
  if (!dQ_out || !dK_out || !dQ || !dK) return ADASPARK_EINVAL;
  if (!qk_rope_args_ok(freq, rot, d, positions, n_axes, sections, magnitude, w_q, w_k, eps))
    return ADASPARK_EINVAL;
  if ((w_q && !Q) || (w_k && !K)) return ADASPARK_EINVAL;
  if (!rows_aligned(dQ_out, dq_ts, dq_hs, dy_dtype) ||
      !rows_aligned(dK_out, dk_ts, dk_hs, dy_dtype) || !aligned(dQ, 16) || !aligned(dK, 16))
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
  b.gq = dQ; b.gk = dK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  b.part = norm ? reinterpret_cast<float*>(ws + align_up(sizeof(WsHeader))) : nullptr;
  int blocks = sms * kBwdBlocksPerSm<false>;
  if (norm)
    blocks = std::min(sms * kBwdBlocksPerSm<true>, kBwdMaxParts);
  else if (n_tokens > blocks * 4 * 2)
    blocks = sms * kBwdLongBlocks;
  blocks = std::min(blocks, (n_tokens + 3) / 4);
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
    e = launch_after("qk_rope_dw", rope_dw_kernel, dim3(2 * d / 8), dim3(1024), 0, s, 1,
                     reinterpret_cast<WsHeader*>(ws), b.part, blocks, d, w_q ? dw_q : nullptr,
                     w_k ? dw_k : nullptr);
  return cuda_status(e);
}

}  // extern "C"
