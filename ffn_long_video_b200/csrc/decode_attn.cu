// Attention of one new token per sequence over a paged key-value cache.
//
// For sequence i of n keys, query head h (KV head h / (hq/hkv)) and z_j = scale q . k_j:
//   out = sum_j exp(z_j - lse) v_j,   lse = log sum_j exp(z_j),   j < n;
// n = 0 (or every z_j = -inf) gives out = 0, lse = -inf.
//
// Bound by the cache's bytes: each key and value is read once for all the query
// heads of its KV head. The work is cut into tiles of keys, and all tiles of all
// (sequence, KV head, group of 8 query heads) runs are laid on one line that the
// blocks share evenly, whatever the lengths: block b of B takes tiles
// [b T / B, (b + 1) T / B). A block keeps the running maximum, sum and output of
// the run it is in; a run that lies in one block is finished there, a cut one
// leaves partial results in the workspace (at most two per block), and a second
// kernel joins them. The cut follows lengths and grid alone, and parts are joined
// in order, so results do not depend on timing.
#include <cmath>

#include "serve.h"

namespace adaspark {

struct DecodeArgs {
  WsHeader* hdr;
  const void* q;
  HeadRows qs;
  const void *kc, *vc;
  CacheRows cs;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  void* out;
  float* lse;                    // or null
  float scale_log2;              // scale * log2(e)
  int32_t n_seqs, max_len, hq, hkv, group, hgroups;  // hgroups: groups of 8 heads per KV head
  int32_t* status;               // [grid] status bits of each block
  int4* joins;                   // [grid] {seq, KV head * hgroups + group, first slot, last slot}
  float* part;                   // [2 grid][8][D + 2]: outputs, maximum (log2), sum
};

constexpr int kDecHeads = 8;     // query heads of a run
constexpr int kDecWarps = 4;
constexpr int kDecStages = 3;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // nothing is read for 0; the 16 bytes become zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Keys of sequence i, 0 for a length the table cannot hold (flagged).
__device__ __forceinline__ int dec_len(const DecodeArgs& a, int i, uint32_t* bits) {
  const int n = a.lens[i];
  if (n >= 0 && n <= a.max_len) return n;
  *bits |= ADASPARK_DEV_BAD_LAYOUT;
  return 0;
}

// Position of a block on the line of tiles.
struct DecSpot {
  int seq, len, tiles;   // sequence, its keys, its tiles per run
  int run;               // KV head * hgroups + group
  int tile;              // tile in the run
};

// Tiles before every sequence: the total, and the sequence that holds tile `at`.
template <int TILE>
__device__ __forceinline__ long long dec_total(const DecodeArgs& a, long long* warp_sum,
                                               long long* before, uint32_t* bits) {
  // thread i sums sequences [i * per, (i + 1) * per)
  const int per = (a.n_seqs + blockDim.x - 1) / blockDim.x;
  const int i0 = min(a.n_seqs, (int)threadIdx.x * per), i1 = min(a.n_seqs, i0 + per);
  long long own = 0;
  for (int i = i0; i < i1; ++i) own += (dec_len(a, i, bits) + TILE - 1) / TILE;
  own *= a.hkv * a.hgroups;
  long long inc = own;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  long long total = 0, base = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  *before = base + inc - own;
  return total;
}

template <typename T, int D>
struct DecShape {
  static constexpr int kKeys = 1024 / (D * (int)sizeof(T)) * 4;  // keys of a warp's stage: 4 KB of K
  static constexpr int kTile = kKeys * kDecWarps;
  static constexpr int kRow = D * (int)sizeof(T) + 16;           // padded row
  static constexpr int kStage = 2 * kKeys * kRow;                // K rows, V rows
  static constexpr int kRing = kDecStages * kStage;              // a warp's stages
  static constexpr int kSmem = kDecWarps * kRing;
};

// What a block knows of the line of tiles.
struct DecLine {
  long long total, B;   // tiles, blocks that share them
  long long u0, u1;     // this block's
};

struct DecShared {
  long long warp_sum[kDecWarps];
  DecSpot first;
  float m[kDecWarps][kDecHeads], l[kDecWarps][kDecHeads];
  uint32_t bits[kDecWarps];
};

// Finds the block's share and its first run; writes the results of sequences
// without keys. All threads; ends with a barrier.
template <typename T, int D>
__device__ __forceinline__ DecLine dec_begin(const DecodeArgs& a, DecShared& sh, uint32_t* bits) {
  using S = DecShape<T, D>;
  const int b = blockIdx.x;
  long long before;
  DecLine L;
  L.total = dec_total<S::kTile>(a, sh.warp_sum, &before, bits);
  // blocks that share the line: each of them has a tile at least
  L.B = min((long long)gridDim.x, L.total);
  L.u0 = b < L.B ? L.total * b / L.B : 0;
  L.u1 = b < L.B ? L.total * (b + 1) / L.B : 0;
  if (L.u0 < L.u1) {
    const int per = (a.n_seqs + blockDim.x - 1) / blockDim.x;
    const int i0 = min(a.n_seqs, (int)threadIdx.x * per), i1 = min(a.n_seqs, i0 + per);
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      const int len = dec_len(a, i, bits), tiles = (len + S::kTile - 1) / S::kTile;
      const long long mine = (long long)tiles * a.hkv * a.hgroups;
      if (L.u0 >= at && L.u0 < at + mine) {
        const int in = (int)(L.u0 - at);
        sh.first = DecSpot{i, len, tiles, in / tiles, in % tiles};
      }
      at += mine;
    }
  }
  for (int i = b; i < a.n_seqs; i += gridDim.x) {
    if (dec_len(a, i, bits) > 0) continue;
    for (int e = threadIdx.x; e < a.hq * D; e += blockDim.x)
      static_cast<T*>(a.out)[(int64_t)i * a.hq * D + e] = from_f32<T>(0.f);
    if (a.lse)
      for (int h = threadIdx.x; h < a.hq; h += blockDim.x)
        a.lse[(int64_t)i * a.hq + h] = -INFINITY;
  }
  __syncthreads();
  return L;
}

// Element offset of a key's row in the cache, -1 for a key that is not there.
// `page` is the table's entry for the key (any value where key >= len).
__device__ __forceinline__ int64_t dec_offset(const DecodeArgs& a, int key, int len, int page,
                                              int kvh, uint32_t* bits) {
  if (key >= len) return -1;
  if (page < 0 || page >= a.cs.n_pages) {
    *bits |= ADASPARK_DEV_BAD_LAYOUT;
    return -1;
  }
  return page * a.cs.ps + (key % a.cs.page_size) * a.cs.ts + kvh * a.cs.hs;
}

// Copies a stage's rows, row r at lane r's offset: consecutive lanes take the
// 16-byte pieces of a row. One commit group, empty when nothing is wanted.
template <typename T, int D>
__device__ __forceinline__ void dec_copy(const DecodeArgs& a, uint8_t* st, int64_t off, bool want) {
  using S = DecShape<T, D>;
  constexpr int per_row = D * (int)sizeof(T) / 16, rows = 32 / per_row;
  const int lane = threadIdx.x & 31, r0 = lane / per_row, piece = lane % per_row;
  if (want) {
#pragma unroll
    for (int r = 0; r < S::kKeys; r += rows) {
      const int64_t ro = __shfl_sync(0xffffffffu, off, r + r0);
      const bool ok = ro >= 0;
      const int64_t byte = (ok ? ro * (int)sizeof(T) : 0) + piece * 16;
      cp_async16(st + (r + r0) * S::kRow + piece * 16, static_cast<const uint8_t*>(a.kc) + byte, ok);
      cp_async16(st + (S::kKeys + r + r0) * S::kRow + piece * 16,
                 static_cast<const uint8_t*>(a.vc) + byte, ok);
    }
  }
  cp_async_commit();
}

// Joins the warps' parts of a run (maxima and sums in sh, outputs [8][D] at the
// start of each warp's ring) and writes its results or the block's partial ones.
// All threads; the caller puts a barrier before and after. Returns the joins
// entry of a cut run that starts in this block.
template <typename T, int D>
__device__ __forceinline__ void dec_end_run(const DecodeArgs& a, const DecShared& sh,
                                            const uint8_t* smem, const DecSpot& at, int n_tiles,
                                            long long u, const DecLine& L, int4* join) {
  using S = DecShape<T, D>;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
  const int heads = min(kDecHeads, a.group - hg * kDecHeads);
  const int h0 = kvh * a.group + hg * kDecHeads;
  const bool whole = at.tile == 0 && n_tiles == at.tiles;
  const int slot = 2 * blockIdx.x + (u == L.u0 ? 0 : 1);
  for (int h = warp; h < heads; h += kDecWarps) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, sh.m[w][h]);
    const float mu = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[E] = {};
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float f = exp2f(sh.m[w][h] - mu);
      ll = fmaf(sh.l[w][h], f, ll);
      const float* ob = reinterpret_cast<const float*>(smem + w * S::kRing);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(ob[h * D + lane * E + e], f, acc[e]);
    }
    if (whole) {
      const float r = 1.f / ll;
      T* op = static_cast<T*>(a.out) + ((int64_t)at.seq * a.hq + h0 + h) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) op[e] = from_f32<T>(ll == 0.f ? 0.f : acc[e] * r);
      if (a.lse && lane == 0)
        a.lse[(int64_t)at.seq * a.hq + h0 + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    } else {
      float* pp = a.part + ((int64_t)slot * kDecHeads + h) * (D + 2);
#pragma unroll
      for (int e = 0; e < E; ++e) pp[lane * E + e] = acc[e];
      if (lane == 0) {
        pp[D] = mm;
        pp[D + 1] = ll;
      }
    }
  }
  if (!whole && at.tile == 0) {
    // the first block of a cut run: its parts are this slot and the first slots of the
    // blocks up to the one that holds the run's last tile
    const long long end = u + at.tiles - 1;
    long long last = end * L.B / L.total;
    while (L.total * (last + 1) / L.B <= end) ++last;
    while (L.total * last / L.B > end) --last;
    *join = make_int4(at.seq, at.run, slot, 2 * (int)last);
  }
}

// Next run on the line.
template <int TILE>
__device__ __forceinline__ void dec_advance(const DecodeArgs& a, DecSpot* at, uint32_t* bits) {
  at->tile = 0;
  if (++at->run < a.hkv * a.hgroups) return;
  at->run = 0;
  do {
    if (++at->seq >= a.n_seqs) return;
    at->len = dec_len(a, at->seq, bits);
    at->tiles = (at->len + TILE - 1) / TILE;
  } while (at->tiles == 0);
}

__device__ __forceinline__ void dec_end(const DecodeArgs& a, DecShared& sh, uint32_t bits,
                                        int4 join) {
  bits = __reduce_or_sync(0xffffffffu, bits);
  if ((threadIdx.x & 31) == 0) sh.bits[threadIdx.x >> 5] = bits;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t v = 0;
    for (int w = 0; w < kDecWarps; ++w) v |= sh.bits[w];
    a.status[blockIdx.x] = (int32_t)v;
    a.joins[blockIdx.x] = join;
  }
}

template <int E>
__device__ __forceinline__ void dec_row(const uint8_t* row, int lane, float (&v)[E]);
template <>
__device__ __forceinline__ void dec_row<4>(const uint8_t* row, int lane, float (&v)[4]) {
  const float4 x = reinterpret_cast<const float4*>(row)[lane];
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
template <>
__device__ __forceinline__ void dec_row<2>(const uint8_t* row, int lane, float (&v)[2]) {
  const float2 x = reinterpret_cast<const float2*>(row)[lane];
  v[0] = x.x; v[1] = x.y;
}

// fp32: each lane holds D / 32 elements of every row and of 8 heads' outputs; a
// warp's keys pass through a ring of stages of its own in shared memory
// (cp.async), so warps run without block barriers inside a run.
template <int D>
__global__ void __launch_bounds__(kDecWarps * 32) decode_simt_kernel(const DecodeArgs a) {
  using T = float;
  using S = DecShape<T, D>;
  constexpr int E = D / 32, KK = S::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DecShared sh;
  __shared__ __align__(16) float pbuf[kDecWarps][KK][kDecHeads];  // read 16 bytes at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependency_release();
  uint32_t bits = 0;
  const DecLine L = dec_begin<T, D>(a, sh, &bits);
  int4 join = make_int4(-1, 0, 0, 0);
  DecSpot at = sh.first;
  uint8_t* ring = smem + warp * S::kRing;
  for (long long u = L.u0; u < L.u1;) {
    const int n_tiles = (int)min((long long)(at.tiles - at.tile), L.u1 - u);
    const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
    const int heads = min(kDecHeads, a.group - hg * kDecHeads);
    const int h0 = kvh * a.group + hg * kDecHeads;
    float q[kDecHeads][E], o[kDecHeads][E];
    float m = -INFINITY, l = 0.f;   // this lane's head: lane % 8
#pragma unroll
    for (int h = 0; h < kDecHeads; ++h) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[h][e] = 0.f;
        o[h][e] = 0.f;
      }
      if (h < heads) {
        const T* p = static_cast<const T*>(a.q) + at.seq * a.qs.ts + (h0 + h) * a.qs.hs;
#pragma unroll
        for (int e = 0; e < E; ++e) q[h][e] = p[lane * E + e];
      }
    }
    const int32_t* pages = a.table + at.seq * a.table_stride;
    const int key0 = at.tile * S::kTile + warp * KK;

    // Rows of stage i into the ring; returns the bits of the rows that are there.
    auto fetch = [&](int i) -> uint32_t {
      const int key = key0 + i * S::kTile + lane;
      int64_t off = -1;
      if (i < n_tiles && lane < KK && key < at.len)
        off = dec_offset(a, key, at.len, pages[key / a.cs.page_size], kvh, &bits);
      dec_copy<T, D>(a, ring + (i % kDecStages) * S::kStage, off, i < n_tiles);
      return __ballot_sync(0xffffffffu, off >= 0);
    };

    uint32_t there[kDecStages];
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) there[i] = fetch(i);
    for (int i = 0; i < n_tiles; ++i) {
      __syncwarp();  // the stage that is fetched into was read by every lane
      const uint32_t next = fetch(i + kDecStages - 1);
      cp_async_wait<kDecStages - 1>();
      __syncwarp();
      const uint32_t here = there[0];
#pragma unroll
      for (int k = 0; k + 1 < kDecStages - 1; ++k) there[k] = there[k + 1];
      there[kDecStages - 2] = next;
      const uint8_t* st = ring + (i % kDecStages) * S::kStage;
      // scores, four keys at a time; lane = key * 8 + head holds one of the 32 sums
      float z[KK / 4];
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < KK / 4; ++g) {
        float d[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x[E];
          dec_row<E>(st + (4 * g + k) * S::kRow, lane, x);
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            float acc = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc = fmaf(q[h][e], x[e], acc);
            d[k * 8 + h] = acc;
          }
        }
        // halve the values while folding the lanes: lane bit w keeps the half with that bit
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) {
#pragma unroll
          for (int j = 0; j < w; ++j) {
            const bool up = lane & w;
            const float keep = up ? d[j + w] : d[j], give = up ? d[j] : d[j + w];
            d[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
          }
        }
        const bool ok = here >> (4 * g + (lane >> 3)) & 1;
        z[g] = ok ? d[0] * a.scale_log2 : -INFINITY;
        top = fmaxf(top, z[g]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float m_new = fmaxf(m, top);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m - m_use);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int g = 0; g < KK / 4; ++g) {
        const float p = exp2f(z[g] - m_use);
        l += p;
        pbuf[warp][4 * g + (lane >> 3)][lane & 7] = p;
      }
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float f = __shfl_sync(0xffffffffu, alpha, h);
#pragma unroll
          for (int e = 0; e < E; ++e) o[h][e] *= f;
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        float x[E];
        dec_row<E>(st + (KK + k) * S::kRow, lane, x);
        const float4 pa = *reinterpret_cast<const float4*>(&pbuf[warp][k][0]);
        const float4 pb = *reinterpret_cast<const float4*>(&pbuf[warp][k][4]);
        const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
          for (int e = 0; e < E; ++e) o[h][e] = fmaf(p[h], x[e], o[h][e]);
      }
    }
    cp_async_wait<0>();
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (lane < 8) {
      sh.m[warp][lane] = m;
      sh.l[warp][lane] = l;
    }
    __syncwarp();
    float* obuf = reinterpret_cast<float*>(ring);  // this warp's ring is at rest
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) obuf[h * D + lane * E + e] = o[h][e];
    __syncthreads();
    dec_end_run<T, D>(a, sh, smem, at, n_tiles, u, L, &join);
    __syncthreads();
    u += n_tiles;
    dec_advance<S::kTile>(a, &at, &bits);
  }
  dec_end(a, sh, bits, join);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const uint8_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], const uint8_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
// Transpose of an 8x8 matrix of 16-bit elements held by the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// c [16 x 8] += A [16 x 16] B [16 x 8], bf16 in, fp32 accumulation.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// bf16: keys fill the rows of a product's tile and 8 query heads its columns,
//   S^T [16 keys x 8 heads] = K Q^T,   O^T [16 d x 8 heads] += V^T P^T,
// so that no part of a tile is padding when a KV head serves 8 query heads (128
// rows of tcgen05 would hold 7 or 8 of them), and a lane's softmax columns are
// its output columns. P goes to the second product as two bf16 parts (high and
// rest: 2^-17 relative), which costs 8 more products per 16 keys and keeps the
// output as near as fp32 weights would. The warp's keys pass through a ring of
// stages of its own (cp.async), the table entry of a stage one step ahead.
template <int D>
__global__ void __launch_bounds__(kDecWarps * 32) decode_mma_kernel(const DecodeArgs a) {
  using T = __nv_bfloat16;
  using S = DecShape<T, D>;
  constexpr int KK = S::kKeys, MT = KK / 16, DT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DecShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  dependency_release();
  uint32_t bits = 0;
  const DecLine L = dec_begin<T, D>(a, sh, &bits);
  int4 join = make_int4(-1, 0, 0, 0);
  DecSpot at = sh.first;
  uint8_t* ring = smem + warp * S::kRing;
  for (long long u = L.u0; u < L.u1;) {
    const int n_tiles = (int)min((long long)(at.tiles - at.tile), L.u1 - u);
    const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
    const int heads = min(kDecHeads, a.group - hg * kDecHeads);
    const int h0 = kvh * a.group + hg * kDecHeads;
    const int32_t* pages = a.table + at.seq * a.table_stride;
    const int key0 = at.tile * S::kTile + warp * KK + lane;  // of this lane's row, stage 0
    auto entry = [&](int i) -> int {
      const int key = key0 + i * S::kTile;
      return i < n_tiles && lane < KK && key < at.len ? pages[key / a.cs.page_size] : 0;
    };
    auto fetch = [&](int i, int page) -> uint32_t {
      const int64_t off = i < n_tiles && lane < KK
                              ? dec_offset(a, key0 + i * S::kTile, at.len, page, kvh, &bits)
                              : -1;
      dec_copy<T, D>(a, ring + (i % kDecStages) * S::kStage, off, i < n_tiles);
      return __ballot_sync(0xffffffffu, off >= 0);
    };
    uint32_t there[kDecStages];
    int page[kDecStages];
#pragma unroll
    for (int i = 0; i < kDecStages; ++i) page[i] = entry(i);
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) there[i] = fetch(i, page[i]);
    int ahead = page[kDecStages - 1];
    // Q^T: column g is head g, rows 2c, 2c + 1 and 8 further of each 16 of d
    uint32_t qf[DT][2];
#pragma unroll
    for (int k = 0; k < DT; ++k) {
      qf[k][0] = qf[k][1] = 0u;
      if (g < heads) {
        const T* p = static_cast<const T*>(a.q) + at.seq * a.qs.ts + (h0 + g) * a.qs.hs + 16 * k +
                     2 * c;
        qf[k][0] = *reinterpret_cast<const uint32_t*>(p);
        qf[k][1] = *reinterpret_cast<const uint32_t*>(p + 8);
      }
    }
    float o[DT][4];
#pragma unroll
    for (int k = 0; k < DT; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1

    for (int i = 0; i < n_tiles; ++i) {
      __syncwarp();  // the stage that is fetched into was read by every lane
      const uint32_t next = fetch(i + kDecStages - 1, ahead);
      ahead = entry(i + kDecStages);
      cp_async_wait<kDecStages - 1>();
      __syncwarp();
      const uint32_t here = there[0];
#pragma unroll
      for (int k = 0; k + 1 < kDecStages - 1; ++k) there[k] = there[k + 1];
      there[kDecStages - 2] = next;
      const uint8_t* st = ring + (i % kDecStages) * S::kStage;
      // scores: rows g and g + 8 of each 16 keys, heads 2c and 2c + 1
      float z[MT][4];
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float s0[4] = {}, s1[4] = {};  // even and odd steps: two shorter chains
        const uint8_t* row = st + (16 * t + (lane & 15)) * S::kRow + (lane >> 4) * 16;
#pragma unroll
        for (int k = 0; k < DT; ++k) {
          uint32_t f[4];
          ldmatrix4(f, row + k * 32);
          if (k & 1)
            mma_16816(s1, f, qf[k][0], qf[k][1]);
          else
            mma_16816(s0, f, qf[k][0], qf[k][1]);
        }
        const bool lo = here >> (16 * t + g) & 1, hi = here >> (16 * t + g + 8) & 1;
        z[t][0] = lo ? (s0[0] + s1[0]) * a.scale_log2 : -INFINITY;
        z[t][1] = lo ? (s0[1] + s1[1]) * a.scale_log2 : -INFINITY;
        z[t][2] = hi ? (s0[2] + s1[2]) * a.scale_log2 : -INFINITY;
        z[t][3] = hi ? (s0[3] + s1[3]) * a.scale_log2 : -INFINITY;
        t0 = fmaxf(t0, fmaxf(z[t][0], z[t][2]));
        t1 = fmaxf(t1, fmaxf(z[t][1], z[t][3]));
      }
#pragma unroll
      for (int w = 4; w <= 16; w <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
      }
      t0 = fmaxf(t0, m0);
      t1 = fmaxf(t1, m1);
      const float u0 = t0 == -INFINITY ? 0.f : t0, u1 = t1 == -INFINITY ? 0.f : t1;
      if (__any_sync(0xffffffffu, t0 != m0 || t1 != m1)) {
        const float f0 = exp2f(m0 - u0), f1 = exp2f(m1 - u1);
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int k = 0; k < DT; ++k) {
          o[k][0] *= f0; o[k][1] *= f1; o[k][2] *= f0; o[k][3] *= f1;
        }
        m0 = t0;
        m1 = t1;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const float p0 = exp2f(z[t][0] - u0), p1 = exp2f(z[t][1] - u1);
        const float p2 = exp2f(z[t][2] - u0), p3 = exp2f(z[t][3] - u1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        const uint32_t ha = pack_bf16x2(p0, p1), hb = pack_bf16x2(p2, p3);
        const uint32_t ra = pack_bf16x2(p0 - __uint_as_float(ha << 16),
                                        p1 - __uint_as_float(ha & 0xffff0000u));
        const uint32_t rb = pack_bf16x2(p2 - __uint_as_float(hb << 16),
                                        p3 - __uint_as_float(hb & 0xffff0000u));
        const uint32_t ph0 = movmatrix(ha), ph1 = movmatrix(hb);
        const uint32_t pr0 = movmatrix(ra), pr1 = movmatrix(rb);
        const uint8_t* row = st + (KK + 16 * t + (lane & 7) + (lane >> 4) * 8) * S::kRow +
                             (lane >> 3 & 1) * 16;
#pragma unroll
        for (int k = 0; k < DT; ++k) {
          uint32_t f[4];
          ldmatrix4_trans(f, row + k * 32);
          mma_16816(o[k], f, ph0, ph1);
          mma_16816(o[k], f, pr0, pr1);
        }
      }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, w);
      l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    if (g == 0) {
      sh.m[warp][2 * c] = m0;
      sh.m[warp][2 * c + 1] = m1;
      sh.l[warp][2 * c] = l0;
      sh.l[warp][2 * c + 1] = l1;
    }
    __syncwarp();
    float* obuf = reinterpret_cast<float*>(ring);  // this warp's ring is at rest
#pragma unroll
    for (int k = 0; k < DT; ++k) {
      obuf[2 * c * D + 16 * k + g] = o[k][0];
      obuf[(2 * c + 1) * D + 16 * k + g] = o[k][1];
      obuf[2 * c * D + 16 * k + g + 8] = o[k][2];
      obuf[(2 * c + 1) * D + 16 * k + g + 8] = o[k][3];
    }
    __syncthreads();
    dec_end_run<T, D>(a, sh, smem, at, n_tiles, u, L, &join);
    __syncthreads();
    u += n_tiles;
    dec_advance<S::kTile>(a, &at, &bits);
  }
  dec_end(a, sh, bits, join);
}

// Joins the parts of a run that was cut: one block per block of the first kernel (the run
// that starts there and ends in a later one) and head. Block (0, 0) collects the status.
template <typename T, int D>
__global__ void __launch_bounds__(D) decode_join_kernel(const DecodeArgs a, int B) {
  dependency_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
    uint32_t v = 0;
    for (int i = threadIdx.x; i < B; i += 32) v |= (uint32_t)a.status[i];
    v = __reduce_or_sync(0xffffffffu, v);
    if (threadIdx.x == 0) {
      a.hdr->status = v;
      a.hdr->detail = v ? 0x9100u : 0u;
    }
  }
  const int4 j = a.joins[blockIdx.x];
  if (j.x < 0) return;
  const int kvh = j.y / a.hgroups, hg = j.y % a.hgroups, h = blockIdx.y;
  if (h >= min(kDecHeads, a.group - hg * kDecHeads)) return;
  auto part = [&](int slot) { return a.part + ((int64_t)slot * kDecHeads + h) * (D + 2); };
  const int n = 1 + (j.w - (j.z & ~1)) / 2;        // slots j.z, then the next blocks' first ones
  auto slot_of = [&](int i) { return i == 0 ? j.z : (j.z & ~1) + 2 * i; };
  float mm = -INFINITY;
  for (int i = 0; i < n; ++i) mm = fmaxf(mm, part(slot_of(i))[D]);
  const float mu = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f, acc = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* p = part(slot_of(i));
    const float f = exp2f(p[D] - mu);
    ll = fmaf(p[D + 1], f, ll);
    acc = fmaf(p[threadIdx.x], f, acc);
  }
  const int64_t row = (int64_t)j.x * a.hq + kvh * a.group + hg * kDecHeads + h;
  static_cast<T*>(a.out)[row * D + threadIdx.x] = from_f32<T>(ll == 0.f ? 0.f : acc / ll);
  if (a.lse && threadIdx.x == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

namespace {

constexpr int kDecMaxBlocks = 148 * 2;

struct DecLayout {
  size_t status, joins, part, total;
};
DecLayout dec_layout(int d) {
  DecLayout L{};
  size_t o = align_up(sizeof(WsHeader));
  L.status = o;
  o = align_up(o + kDecMaxBlocks * sizeof(int32_t));
  L.joins = o;
  o = align_up(o + kDecMaxBlocks * sizeof(int4));
  L.part = o;
  o = align_up(o + (size_t)kDecMaxBlocks * 2 * kDecHeads * (d + 2) * sizeof(float));
  L.total = o;
  return L;
}

template <typename T, int D>
cudaError_t launch_decode(const DecodeArgs& a, void (*kernel)(DecodeArgs), int sms,
                          cudaStream_t s) {
  using S = DecShape<T, D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  // no more blocks than tiles the tables can hold
  const int64_t tiles = (int64_t)a.n_seqs * a.hkv * a.hgroups *
                        (((int64_t)a.max_len + S::kTile - 1) / S::kTile);
  int64_t grid = 2 * (int64_t)sms;
  if (grid > kDecMaxBlocks) grid = kDecMaxBlocks;
  if (grid > tiles) grid = tiles;
  const cudaError_t r = launch("decode_attn", kernel, dim3((unsigned)grid), dim3(kDecWarps * 32),
                               S::kSmem, s, a);
  if (r != cudaSuccess) return r;
  const int heads = a.group < kDecHeads ? a.group : kDecHeads;
  return launch_after("decode_join", decode_join_kernel<T, D>, dim3((unsigned)grid, heads), dim3(D),
                      0, s, a, (int)grid);
}

}  // namespace
}  // namespace adaspark

using namespace adaspark;

extern "C" {

size_t adaspark_decode_attn_workspace(int n_seqs, int hq, int hkv, int d, int dtype) {
  if (n_seqs < 1 || !head_sizes_ok(hq, hkv, d, dtype)) return 0;
  return dec_layout(d).total;
}

int adaspark_decode_attn(const void* Q, int64_t q_ts, int64_t q_hs, const void* k_cache,
                         const void* v_cache, int64_t c_ps, int64_t c_ts, int64_t c_hs,
                         int n_pages, int page_size, int dtype, const int32_t* block_table,
                         int64_t table_stride, int max_pages, const int32_t* seq_lens, int n_seqs,
                         int hq, int hkv, int d, float scale, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!Q || !block_table || !seq_lens || !out || !workspace) return ADASPARK_EINVAL;
  if (n_seqs < 1 || max_pages < 1 || !head_sizes_ok(hq, hkv, d, dtype)) return ADASPARK_EINVAL;
  if (!std::isfinite(scale)) return ADASPARK_EINVAL;
  const CacheRows cs{c_ps, c_ts, c_hs, n_pages, page_size};
  if (!cache_ok(k_cache, v_cache, cs, hkv, d, dtype)) return ADASPARK_EINVAL;
  if ((int64_t)max_pages * page_size > INT32_MAX - 1024) return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return ADASPARK_EINVAL;
  if (!aligned(workspace, kAlign) ||
      workspace_bytes < adaspark_decode_attn_workspace(n_seqs, hq, hkv, d, dtype))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  const DecLayout L = dec_layout(d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeArgs a{};
  a.hdr = reinterpret_cast<WsHeader*>(ws);
  a.q = Q; a.qs = {q_ts, q_hs};
  a.kc = k_cache; a.vc = v_cache; a.cs = cs;
  a.table = block_table; a.table_stride = table_stride; a.lens = seq_lens;
  a.out = out; a.lse = lse;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  a.n_seqs = n_seqs; a.max_len = max_pages * page_size;
  a.hq = hq; a.hkv = hkv; a.group = hq / hkv;
  a.hgroups = (a.group + kDecHeads - 1) / kDecHeads;
  a.status = reinterpret_cast<int32_t*>(ws + L.status);
  a.joins = reinterpret_cast<int4*>(ws + L.joins);
  a.part = reinterpret_cast<float*>(ws + L.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == ADASPARK_BF16)
    return cuda_status(
        d == 128 ? launch_decode<__nv_bfloat16, 128>(a, decode_mma_kernel<128>, sms, s)
                 : launch_decode<__nv_bfloat16, 64>(a, decode_mma_kernel<64>, sms, s));
  return cuda_status(d == 128 ? launch_decode<float, 128>(a, decode_simt_kernel<128>, sms, s)
                              : launch_decode<float, 64>(a, decode_simt_kernel<64>, sms, s));
}

}  // extern "C"
