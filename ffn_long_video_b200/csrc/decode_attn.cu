// Attention of one new token per sequence over a paged key-value cache.
//
// For sequence i of n keys, query head h (KV head h / (hq/hkv)) and z_j = scale q . k_j:
//   out = sum_j exp(z_j - lse) v_j,   lse = log sum_j exp(z_j),   j < n;
// n = 0 (or every z_j = -inf) gives out = 0, lse = -inf.
//
// Bound by the cache's bytes: each key and value is read once for all the query
// heads of its KV head. The work is cut into tiles of keys, and all tiles of all
// (sequence, KV head, group of query heads) runs are laid on one line that the
// blocks share evenly, whatever the lengths: block b of B takes tiles
// [b T / B, (b + 1) T / B). A block keeps the running maximum, sum and output of
// the run it is in; a run that lies in one block is finished there, a cut one
// leaves partial results in the workspace (at most two per block), and a second
// kernel joins them. The cut follows lengths and grid alone, and parts are joined
// in order, so results do not depend on timing.
#include <algorithm>
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
  int32_t n_seqs, max_len, hq, hkv, group, hgroups;  // hgroups: runs per KV head
  int32_t by_run;
  int32_t in_page;               // a page holds a whole number of stages
  int32_t tile_pages, tile_rest; // pages and tokens beyond them that a tile spans
  int32_t* status;               // [grid] status bits of each block
  int4* joins;                   // {seq, KV head * hgroups + group, first slot, last slot} or -1:
                                 // of each run (by_run: there are no more than blocks), or of
                                 // the cut run that starts in each block
  float* part;                   // [2 grid][H][D + 2]: outputs, maximum (log2), sum
};

constexpr int kDecMaxHeads = 16;
constexpr int kDecWarps = 4;
constexpr int kDecMaxBlocks = 148 * 3;
constexpr int kDecCluster = 8;   // blocks that join through shared memory, at most
constexpr float kLn2 = 0.69314718055994530942f;

// Sizes of a warp's work: a tile is kKeys keys of each of the block's warps, a
// stage a warp's share of it, a ring the stages it has in flight. bf16 rows are
// padded so that the 8 rows of a matrix load fall on different banks.
template <typename T_, int D_, int H_>
struct DecShape {
  using T = T_;
  static constexpr int D = D_, H = H_;                        // H: query heads of a run
  static constexpr int kKeys = 4096 / (D * (int)sizeof(T));  // 4 KB of K
  static constexpr int kTile = kKeys * kDecWarps;
  static constexpr int kRow = D * (int)sizeof(T) + (sizeof(T) == 2 ? 16 : 0);
  static constexpr int kStage = 2 * kKeys * kRow;            // K rows, V rows
  static constexpr int kStages = 2;
  // Blocks per SM (registers and shared memory allow no more): fp32 with up to 4 heads 3 (30
  // sequences up to 12829 keys, 6 heads on 3: 52 us at 3, 67 at 2), with more 2; bf16 with up
  // to 8 heads 3, with 16 2.
  static constexpr int kBlocks = H <= (sizeof(T) == 2 ? 8 : 4) ? 3 : 2;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSmem = kDecWarps * kRing;
  static constexpr uint32_t kAll = 0xffffffffu >> (32 - kKeys);
};

// Position of a block on the line of tiles.
struct DecSpot {
  int seq, len, tiles;   // sequence, its keys, its tiles per run
  int run;               // KV head * hgroups + group
  int tile;              // tile in the run
};

// The line of tiles and a block's share of it. The host keeps the tiles that the
// tables can hold below 2^31, so all of this fits 32 bits.
struct DecLine {
  int total, B;         // tiles, blocks that share them: each of them has one at least
  int u0, u1;           // this block's
  int each, rest;       // total / B, total % B: the first `rest` blocks take one more

  __device__ __forceinline__ int start(int b) const { return b * each + min(b, rest); }
  __device__ __forceinline__ int owner(int tile) const {
    const int cut = rest * (each + 1);
    return tile < cut ? tile / (each + 1) : rest + (tile - cut) / each;
  }
};

struct DecShared {
  int warp_sum[kDecWarps];
  DecSpot first;
  float m[kDecWarps][kDecMaxHeads], l[kDecWarps][kDecMaxHeads];
  uint32_t bits[kDecWarps];
};

// Keys of sequence i, 0 for a length the table cannot hold (flagged).
__device__ __forceinline__ int dec_len(const DecodeArgs& a, int i, uint32_t* bits) {
  const int n = a.lens[i];
  if (n >= 0 && n <= a.max_len) return n;
  *bits |= ADASPARK_DEV_BAD_LAYOUT;
  return 0;
}

// Finds the block's share and its first run; writes the results of sequences
// without keys. All threads; ends with a barrier.
template <class S>
__device__ __forceinline__ DecLine dec_begin(const DecodeArgs& a, DecShared& sh, uint32_t* bits) {
  using T = typename S::T;
  constexpr int D = S::D;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int runs = a.hkv * a.hgroups;
  // thread i sums the tiles of sequences [i * per, (i + 1) * per)
  const int per = (a.n_seqs + kDecWarps * 32 - 1) / (kDecWarps * 32);
  const int i0 = min(a.n_seqs, (int)threadIdx.x * per), i1 = min(a.n_seqs, i0 + per);
  int own = 0, len = 0;
  for (int i = i0; i < i1; ++i) {
    len = dec_len(a, i, bits);
    own += (len + S::kTile - 1) / S::kTile * runs;
  }
  int inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sh.warp_sum[warp] = inc;
  __syncthreads();
  DecLine L;
  L.total = 0;
  int before = inc - own;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    L.total += sh.warp_sum[w];
  }
  L.B = min((int)gridDim.x, L.total);
  L.each = L.B ? L.total / L.B : 0;
  L.rest = L.total - L.B * L.each;
  L.u0 = b < L.B ? L.start(b) : 0;
  L.u1 = b < L.B ? L.start(b + 1) : 0;
  if (L.u0 < L.u1 && L.u0 >= before && L.u0 < before + own) {
    for (int i = i0, at = before; i < i1; ++i) {
      if (per > 1) len = dec_len(a, i, bits);
      const int tiles = (len + S::kTile - 1) / S::kTile, mine = tiles * runs;
      if (L.u0 < at + mine) {
        const int in = L.u0 - at;
        sh.first = DecSpot{i, len, tiles, in / tiles, in % tiles};
        break;
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
    if (a.by_run)
      for (int r = threadIdx.x; r < runs; r += blockDim.x) a.joins[i * runs + r].x = -1;
  }
  __syncthreads();
  return L;
}

// The block's status word; block 0 writes the header that counts them. All threads.
__device__ __forceinline__ void dec_status(const DecodeArgs& a, DecShared& sh, uint32_t bits) {
  bits = __reduce_or_sync(0xffffffffu, bits);
  if ((threadIdx.x & 31) == 0) sh.bits[threadIdx.x >> 5] = bits;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t v = 0;
    for (int w = 0; w < kDecWarps; ++w) v |= sh.bits[w];
    a.status[blockIdx.x] = (int32_t)v;
    if (blockIdx.x == 0) {
      a.hdr->status = a.hdr->detail = 0;
      a.hdr->n_block_status = gridDim.x;
    }
  }
}

// Next run on the line (seq = n_seqs behind the last one).
template <class S>
__device__ __forceinline__ void dec_next_run(const DecodeArgs& a, DecSpot* at, uint32_t* bits) {
  at->tile = 0;
  if (++at->run < a.hkv * a.hgroups) return;
  at->run = 0;
  do {
    if (++at->seq >= a.n_seqs) return;
    at->len = dec_len(a, at->seq, bits);
    at->tiles = (at->len + S::kTile - 1) / S::kTile;
  } while (at->tiles == 0);
}

// A stage's row of this lane, its table entry on the way.
struct DecRow {
  int page, in_page, kvh;   // in_page: token in the page, -1: no key
};

// The walk of the copies, ahead of the arithmetic: the lane's key, its page and
// its place there, moved on without a division.
template <class S>
struct DecWalk {
  DecSpot at;
  int key, page, in_page, kvh;
  int page0, in_page0;       // of the lane's key in a run's first tile
  const int32_t* table;

  __device__ __forceinline__ DecWalk(const DecodeArgs& a, const DecSpot& first) : at(first) {
    const int own = (threadIdx.x >> 5) * S::kKeys + (threadIdx.x & 31);
    page0 = own / a.cs.page_size;
    in_page0 = own - page0 * a.cs.page_size;
    key = at.tile * S::kTile + own;
    page = key / a.cs.page_size;
    in_page = key - page * a.cs.page_size;
    kvh = at.run / a.hgroups;
    table = a.table + at.seq * a.table_stride;
  }
  __device__ __forceinline__ DecRow row() const {
    DecRow r{0, -1, kvh};
    if ((threadIdx.x & 31) < S::kKeys && key < at.len) {
      r.page = table[page];
      r.in_page = in_page;
    }
    return r;
  }
  __device__ __forceinline__ void next(const DecodeArgs& a, uint32_t* bits) {
    if (++at.tile < at.tiles) {
      key += S::kTile;
      page += a.tile_pages;
      in_page += a.tile_rest;
      if (in_page >= a.cs.page_size) {
        in_page -= a.cs.page_size;
        ++page;
      }
      return;
    }
    dec_next_run<S>(a, &at, bits);
    key = (threadIdx.x >> 5) * S::kKeys + (threadIdx.x & 31);
    page = page0;
    in_page = in_page0;
    kvh = at.run / a.hgroups;
    table = a.table + at.seq * a.table_stride;
  }
};

// Copies a stage's rows into shared memory (one commit group, empty when nothing
// is wanted) and returns the bits of the rows that are there; absent rows become
// zeros. Consecutive lanes take the 16-byte pieces of a row.
template <class S>
__device__ __forceinline__ uint32_t dec_copy(const DecodeArgs& a, uint8_t* st, const DecRow& r,
                                             bool want, uint32_t* bits) {
  constexpr int es = (int)sizeof(typename S::T), per_row = S::D * es / 16, rows = 32 / per_row;
  const int lane = threadIdx.x & 31, r0 = lane / per_row, piece = lane % per_row;
  uint32_t there = 0;
  if (want) {
    int64_t off = -1;
    if (r.in_page >= 0) {
      if (r.page >= 0 && r.page < a.cs.n_pages)
        off = r.page * a.cs.ps + r.in_page * a.cs.ts + r.kvh * a.cs.hs;
      else
        *bits |= ADASPARK_DEV_BAD_LAYOUT;
    }
    there = __ballot_sync(0xffffffffu, off >= 0);
    uint8_t* kd = st + r0 * S::kRow + piece * 16;
    uint8_t* vd = kd + S::kKeys * S::kRow;
    if (a.in_page && there == S::kAll) {
      // a page holds all rows: they lie ts apart and one offset serves (fp32, 24 sequences of
      // 20000 to 30001 keys, one call after another: 443 us, 459 with an exchange per row;
      // bf16 the same either way)
      const int64_t o0 = __shfl_sync(0xffffffffu, off, 0);
      const int64_t byte = (o0 + r0 * a.cs.ts) * es + piece * 16, step = rows * a.cs.ts * es;
      const uint8_t* ks = static_cast<const uint8_t*>(a.kc) + byte;
      const uint8_t* vs = static_cast<const uint8_t*>(a.vc) + byte;
#pragma unroll
      for (int i = 0; i < S::kKeys; i += rows) {
        cp_async16(kd + i * S::kRow, ks, true);
        cp_async16(vd + i * S::kRow, vs, true);
        ks += step;
        vs += step;
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::kKeys; i += rows) {
        const int64_t ro = __shfl_sync(0xffffffffu, off, i + r0);
        const bool ok = ro >= 0;
        const int64_t byte = (ok ? ro * es : 0) + piece * 16;
        cp_async16(kd + i * S::kRow, static_cast<const uint8_t*>(a.kc) + byte, ok);
        cp_async16(vd + i * S::kRow, static_cast<const uint8_t*>(a.vc) + byte, ok);
      }
    }
  }
  cp_async_commit();
  return there;
}

// Ends a run, or the block's share of one: joins the warps' maxima, sums and
// outputs and writes results or partial ones. The outputs pass through the stage
// that each warp has just used (`used`; [H][D + 4] floats), the other stages are
// being filled for the tiles to come. All threads; ends with a barrier. `u`: tile
// on the line where the block's share of the run began; `from`: that tile in the run.
template <class M>
__device__ __forceinline__ void dec_end_run(const DecodeArgs& a, DecShared& sh, M& math,
                                            uint8_t* smem, int used, const DecSpot& at, int from,
                                            int u, const DecLine& L, int4* join) {
  using S = typename M::S;
  using T = typename S::T;
  constexpr int D = S::D, E = D / 32;
  static_assert(S::H * (D + 4) * 4 <= S::kStage, "");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
  const int heads = min(S::H, a.group - hg * S::H);
  const int h0 = kvh * a.group + hg * S::H;
  const bool whole = from == 0 && at.tile + 1 == at.tiles;
  const int slot = 2 * blockIdx.x + (u == L.u0 ? 0 : 1);
  math.sums(sh.m[warp], sh.l[warp]);
  __syncwarp();
  math.outputs(reinterpret_cast<float*>(smem + warp * S::kRing + used * S::kStage));
  __syncthreads();
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
      const float* o = reinterpret_cast<const float*>(smem + w * S::kRing + used * S::kStage);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(o[h * (D + 4) + 32 * e + lane], f, acc[e]);
    }
    const int64_t row = (int64_t)at.seq * a.hq + h0 + h;
    if (whole) {
      const float r = 1.f / ll;
#pragma unroll
      for (int e = 0; e < E; ++e)
        static_cast<T*>(a.out)[row * D + 32 * e + lane] =
            from_f32<T>(ll == 0.f ? 0.f : acc[e] * r);
      if (a.lse && lane == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    } else {
      float* pp = a.part + ((int64_t)slot * S::H + h) * (D + 2);
#pragma unroll
      for (int e = 0; e < E; ++e) pp[32 * e + lane] = acc[e];
      if (lane == 0) {
        pp[D] = mm;
        pp[D + 1] = ll;
      }
    }
  }
  if (from == 0) {
    // the first block of a run; the parts of a cut one are this slot and the first slots of
    // the blocks up to the one that holds the run's last tile
    const int4 j = whole ? make_int4(-1, 0, 0, 0)
                         : make_int4(at.seq, at.run, slot, 2 * L.owner(u + at.tiles - 1));
    if (!whole) *join = j;
    if (a.by_run && threadIdx.x == 0) a.joins[at.seq * a.hkv * a.hgroups + at.run] = j;
  }
  __syncthreads();
}

// The walk along the line. Each warp's keys pass through a ring of stages of its
// own in shared memory (cp.async), so warps run without block barriers inside a
// run; the copies run on across runs, and a stage's table entries are fetched a
// step before its copies are issued. M: the arithmetic (a run's queries,
// maxima, sums and outputs in registers).
template <class M>
__global__ void __launch_bounds__(kDecWarps * 32, M::S::kBlocks) decode_kernel(const DecodeArgs a) {
  using S = typename M::S;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DecShared sh;
  __shared__ typename M::Shared msh;
  const int warp = threadIdx.x >> 5;
  dependency_wait();
  uint32_t bits = 0;
  const DecLine L = dec_begin<S>(a, sh, &bits);
  int4 join = make_int4(-1, 0, 0, 0);
  const int steps = L.u1 - L.u0;
  if (steps > 0) {
    DecSpot at = sh.first;
    DecWalk<S> ahead(a, at);   // at step min(i + kStages, steps) when step i begins
    uint8_t* ring = smem + warp * S::kRing;
    uint32_t there[S::kStages - 1];
    DecRow row[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) {
      if (i < steps) row[i] = ahead.row();
      if (i + 1 < steps) ahead.next(a, &bits);
    }
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i)
      there[i] = dec_copy<S>(a, ring + i * S::kStage, row[i], i < steps, &bits);
    DecRow next = row[S::kStages - 1];
    M math(a, msh);
    math.begin(at);
    int from = at.tile, u = L.u0, stage = 0;
    for (int i = 0; i < steps; ++i) {
      __syncwarp();  // the stage that is copied into was read by every lane
      const uint32_t coming =
          dec_copy<S>(a, ring + (stage == 0 ? S::kStages - 1 : stage - 1) * S::kStage, next,
                      i + S::kStages - 1 < steps, &bits);
      if (i + S::kStages < steps) {
        next = ahead.row();
        if (i + S::kStages + 1 < steps) ahead.next(a, &bits);
      }
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      math.tile(ring + stage * S::kStage, there[0]);
#pragma unroll
      for (int k = 0; k < S::kStages - 2; ++k) there[k] = there[k + 1];
      there[S::kStages - 2] = coming;
      if (at.tile + 1 == at.tiles || i + 1 == steps) {
        dec_end_run(a, sh, math, smem, stage, at, from, u, L, &join);
        u = L.u0 + i + 1;
        from = 0;
        if (i + 1 < steps) {
          dec_next_run<S>(a, &at, &bits);
          math.begin(at);
        }
      } else {
        ++at.tile;
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
  }
  dec_status(a, sh, bits);
  if (threadIdx.x == 0 && !a.by_run) a.joins[blockIdx.x] = join;
}

// Address of a peer block's shared memory, loads from it, and the cluster's barrier.
__device__ __forceinline__ uint32_t peer_smem(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_load(uint32_t address) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(address) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Few short runs: a cluster of blocks per run (no line to lay out), each with an
// even share of its tiles; the parts are joined through the blocks' shared memory
// and there is no second kernel (one sequence of 500 keys, 28 heads on 4, one call
// after another: 5.1 us; 6.5 along the line, under a table of 4113 pages of 16). All
// branches around the barriers go
// by the sequence's length, which the cluster shares.
template <class M>
__global__ void __launch_bounds__(kDecWarps * 32, M::S::kBlocks)
    decode_cluster_kernel(const DecodeArgs a, int C) {
  using S = typename M::S;
  using T = typename S::T;
  constexpr int D = S::D, E = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DecShared sh;
  __shared__ typename M::Shared msh;
  __shared__ float part[S::H][D + 2];   // this block's outputs, maxima, sums
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % C, runs = a.hkv * a.hgroups;
  uint32_t bits = 0;
  DecSpot at;
  at.seq = blockIdx.x / C / runs;
  at.run = blockIdx.x / C - at.seq * runs;
  at.len = dec_len(a, at.seq, &bits);
  at.tiles = (at.len + S::kTile - 1) / S::kTile;
  const int heads = min(S::H, a.group - at.run % a.hgroups * S::H);
  const int64_t row0 = (int64_t)at.seq * a.hq + at.run / a.hgroups * a.group +
                       at.run % a.hgroups * S::H;
  if (at.len == 0) {
    if (rank == 0) {
      for (int e = threadIdx.x; e < heads * D; e += kDecWarps * 32)
        static_cast<T*>(a.out)[row0 * D + e] = from_f32<T>(0.f);
      if (a.lse && threadIdx.x < heads) a.lse[row0 + threadIdx.x] = -INFINITY;
    }
  } else {
    at.tile = at.tiles * rank / C;
    const int steps = at.tiles * (rank + 1) / C - at.tile;
    uint8_t* ring = smem + warp * S::kRing;
    DecWalk<S> ahead(a, at);
    uint32_t there[S::kStages - 1];
    DecRow row[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) {
      if (i < steps) row[i] = ahead.row();
      if (i + 1 < steps) ahead.next(a, &bits);
    }
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i)
      there[i] = dec_copy<S>(a, ring + i * S::kStage, row[i], i < steps, &bits);
    DecRow next = row[S::kStages - 1];
    M math(a, msh);
    math.begin(at);
    int stage = 0;
    for (int i = 0; i < steps; ++i) {
      __syncwarp();
      const uint32_t coming =
          dec_copy<S>(a, ring + (stage == 0 ? S::kStages - 1 : stage - 1) * S::kStage, next,
                      i + S::kStages - 1 < steps, &bits);
      if (i + S::kStages < steps) {
        next = ahead.row();
        if (i + S::kStages + 1 < steps) ahead.next(a, &bits);
      }
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      math.tile(ring + stage * S::kStage, there[0]);
#pragma unroll
      for (int k = 0; k < S::kStages - 2; ++k) there[k] = there[k + 1];
      there[S::kStages - 2] = coming;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    // the warps' parts into the block's; nothing is in flight any more
    math.sums(sh.m[warp], sh.l[warp]);
    __syncwarp();
    math.outputs(reinterpret_cast<float*>(ring));
    __syncthreads();
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
        const float* o = reinterpret_cast<const float*>(smem + w * S::kRing);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(o[h * (D + 4) + 32 * e + lane], f, acc[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) part[h][32 * e + lane] = acc[e];
      if (lane == 0) {
        part[h][D] = mm;
        part[h][D + 1] = ll;
      }
    }
    cluster_barrier();
    // the blocks' parts, in order: head h by block h % C, warp h / C
    for (int h = rank + C * warp; h < heads; h += C * kDecWarps) {
      const uint32_t peer = peer_smem(part[h], min(lane, C - 1));
      float m = peer_load(peer + D * 4), l = peer_load(peer + D * 4 + 4);
      if (lane >= C) {
        m = -INFINITY;
        l = 0.f;
      }
      const float mm = warp_max(m), mu = mm == -INFINITY ? 0.f : mm;
      const float f = lane < C ? exp2f(m - mu) : 0.f, ll = warp_sum(l * f);
      float acc[E] = {};
      for (int p = 0; p < C; ++p) {
        const uint32_t from = peer_smem(part[h], p);
        const float w = __shfl_sync(0xffffffffu, f, p);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(peer_load(from + (32 * e + lane) * 4), w, acc[e]);
      }
      const float r = 1.f / ll;
#pragma unroll
      for (int e = 0; e < E; ++e)
        static_cast<T*>(a.out)[(row0 + h) * D + 32 * e + lane] =
            from_f32<T>(ll == 0.f ? 0.f : acc[e] * r);
      if (a.lse && lane == 0) a.lse[row0 + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
    cluster_barrier();  // no block leaves while another reads its part
  }
  dec_status(a, sh, bits);
}

// fp32 on the CUDA cores, in packed pairs (two multiply-adds per instruction).
// Scores: 8 lanes share a key (16 or 8 elements each, queries from shared memory,
// two keys at a time), 4 keys side by side; exchanges leave lane j of them with head
// j % HF, HF the next power of two (heads from H on are zeros). Outputs: a lane holds
// D / 32 elements of H heads. Weights pass through shared memory, written twice as a
// pair so that they load as one. Outputs and
// sums are kept in two levels (kFlush tiles, then all): one chain of 2400 keys
// had twice the error. 24 sequences of 20000 to 30001 keys, 28 heads on 4: 390 us
// (floor 384) while the clocks hold; one call after another the power limit lowers
// them and it takes 420 to 433 (441 to 448 in runs of 8 with one head empty).
template <int D, int H>
struct DecFp32 {
  using S = DecShape<float, D, H>;
  static constexpr int E2 = D / 64, KK = S::kKeys, kFlush = 8;
  static constexpr int HF = H <= 2 ? 2 : H <= 4 ? 4 : 8, HP = (H + 1) / 2 * 2;
  struct Shared {
    __align__(16) float q[H][D];
    __align__(16) float2 p[kDecWarps][KK][HP];
  };
  const DecodeArgs& a;
  Shared& sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kg = lane >> 3, j = lane & 7;
  F2 o[H][E2], om[H][E2];
  float m, l, lm;  // this lane's head: j % HF
  int n;

  __device__ __forceinline__ DecFp32(const DecodeArgs& a_, Shared& sh_) : a(a_), sh(sh_) {}

  __device__ __forceinline__ static void lds(const void* p, F2& x, F2& y) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    x.v = v.x;
    y.v = v.y;
  }

  // All threads, at a point where no warp reads the queries of the run before.
  __device__ __forceinline__ void begin(const DecSpot& at) {
    const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
    const int heads = min(H, a.group - hg * H);
    const float* q = static_cast<const float*>(a.q) + at.seq * a.qs.ts +
                     (int64_t)(kvh * a.group + hg * H) * a.qs.hs;
    for (int e = threadIdx.x; e < H * D; e += kDecWarps * 32)
      sh.q[e / D][e % D] = e / D < heads ? q[e / D * a.qs.hs + e % D] : 0.f;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < E2; ++e) o[h][e] = om[h][e] = f2(0.f, 0.f);
    m = -INFINITY;
    l = lm = 0.f;
    n = 0;
  }

  __device__ __forceinline__ void tile(const uint8_t* st, uint32_t here) {
    float z[KK / 4];  // of key 4 g + kg and head j % HF
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < KK / 4; g += 2) {
      F2 acc[2][H];
#pragma unroll
      for (int h = 0; h < H; ++h) acc[0][h] = acc[1][h] = f2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        F2 ka, kb, kc, kd;
        lds(st + (4 * g + kg) * S::kRow + 16 * (j + 8 * c), ka, kb);
        lds(st + (4 * g + 4 + kg) * S::kRow + 16 * (j + 8 * c), kc, kd);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          F2 qa, qb;
          lds(&sh.q[h][4 * (j + 8 * c)], qa, qb);
          acc[0][h] = fma2(ka, qa, acc[0][h]);
          acc[0][h] = fma2(kb, qb, acc[0][h]);
          acc[1][h] = fma2(kc, qa, acc[1][h]);
          acc[1][h] = fma2(kd, qb, acc[1][h]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[HF] = {};
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float2 v = unpack(acc[x][h]);
          d[h] = v.x + v.y;
        }
        // fold the lanes, halving the values while there are more than one: lane bit w keeps
        // the half with that bit
#pragma unroll
        for (int w = 4; w >= 1; w >>= 1) {
          if (w >= HF) {
#pragma unroll
            for (int k = 0; k < HF; ++k) d[k] += __shfl_xor_sync(0xffffffffu, d[k], w);
          } else {
#pragma unroll
            for (int k = 0; k < w; ++k) {
              const bool up = lane & w;
              const float keep = up ? d[k + w] : d[k], give = up ? d[k] : d[k + w];
              d[k] = keep + __shfl_xor_sync(0xffffffffu, give, w);
            }
          }
        }
        const bool ok = here >> (4 * (g + x) + kg) & 1;
        z[g + x] = ok ? d[0] * a.scale_log2 : -INFINITY;
        top = fmaxf(top, z[g + x]);
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    const float m_new = fmaxf(m, top);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    if (__any_sync(0xffffffffu, m_new != m)) {
      const float alpha = exp2f(m - m_use);
      m = m_new;
      l *= alpha;
      lm *= alpha;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float f = __shfl_sync(0xffffffffu, alpha, h);
        const F2 ff = f2(f, f);
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          o[h][e] = mul2(o[h][e], ff);
          om[h][e] = mul2(om[h][e], ff);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < KK / 4; ++g) {
      const float p = exp2f(z[g] - m_use);
      l += p;
      if (j < H) sh.p[warp][4 * g + kg][j] = make_float2(p, p);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const uint8_t* row = st + (KK + k) * S::kRow + lane * (8 * E2);
      F2 x[E2];
      if (E2 == 2)
        lds(row, x[0], x[E2 - 1]);
      else
        x[0].v = *reinterpret_cast<const unsigned long long*>(row);
#pragma unroll
      for (int h = 0; h < H; h += 2) {
        F2 pa, pb;
        lds(&sh.p[warp][k][h], pa, pb);
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          o[h][e] = fma2(pa, x[e], o[h][e]);
          if (h + 1 < H) o[(h + 1) % H][e] = fma2(pb, x[e], o[(h + 1) % H][e]);
        }
      }
    }
    if (++n == kFlush) flush();
  }

  __device__ __forceinline__ void flush() {
    n = 0;
    lm += l;
    l = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        om[h][e] = add2(om[h][e], o[h][e]);
        o[h][e] = f2(0.f, 0.f);
      }
  }

  __device__ __forceinline__ void sums(float* ms, float* ls) {
    flush();
    lm += __shfl_xor_sync(0xffffffffu, lm, 8);
    lm += __shfl_xor_sync(0xffffffffu, lm, 16);
    if (lane < H) {
      ms[lane] = m;
      ls[lane] = lm;
    }
  }
  __device__ __forceinline__ void outputs(float* out) const {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < E2; ++e)
        *reinterpret_cast<float2*>(&out[h * (D + 4) + lane * 2 * E2 + 2 * e]) = unpack(om[h][e]);
  }
};

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

// bf16: keys fill the rows of a product's tile and query heads its columns,
//   S^T [16 keys x 8 heads] = K Q^T,   O^T [16 d x 8 heads] += V^T P^T,
// so that no part of a tile is padding when a KV head serves 8 query heads (the
// 128 rows of a tcgen05 tile would hold 7 or 8 of them), and a lane's softmax
// columns are its output columns. NT = 2: up to 16 heads, each load of a key feeds
// two products. P goes to the second product as two bf16 parts (high and rest:
// 2^-17 relative), which costs 8 more products per 16 keys; with one, each weight
// would be off by up to half a step of bf16. With two, 0.2 % of the outputs of the 61
// sequences below round to a neighbour of the rounded exact value, 0.1 % with fp32
// weights; the error against 64 bits is the rounding's, 1.671e-3, either way.
// 61 sequences up to 9001 keys, 16 heads on 2 of 128: 54.4 us (floor 44.3); one of
// 65793, 28 on 4: 30.6 us with its join (floor 20.9).
template <int D, int NT>
struct DecBf16 {
  using S = DecShape<__nv_bfloat16, D, 8 * NT>;
  static constexpr int KK = S::kKeys, MT = KK / 16, DT = D / 16;
  struct Shared {};
  const DecodeArgs& a;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint32_t qf[NT][DT][2];
  float o[NT][DT][4];
  float m[NT][2], l[NT][2];  // heads 8 n + 2c, 2c + 1

  __device__ __forceinline__ DecBf16(const DecodeArgs& a_, Shared&) : a(a_) {}

  __device__ __forceinline__ void begin(const DecSpot& at) {
    const int kvh = at.run / a.hgroups, hg = at.run % a.hgroups;
    const int heads = min(S::H, a.group - hg * S::H);
    // Q^T: column g is head g, rows 2c, 2c + 1 and 8 further of each 16 of d
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + at.seq * a.qs.ts +
                             (int64_t)(kvh * a.group + hg * S::H + g) * a.qs.hs + 2 * c;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool there = 8 * n + g < heads;
      const __nv_bfloat16* p = q + (int64_t)8 * n * a.qs.hs;
#pragma unroll
      for (int k = 0; k < DT; ++k) {
        qf[n][k][0] = there ? *reinterpret_cast<const uint32_t*>(p + 16 * k) : 0u;
        qf[n][k][1] = there ? *reinterpret_cast<const uint32_t*>(p + 16 * k + 8) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
      }
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const uint8_t* st, uint32_t here) {
    // scores: rows g and g + 8 of each 16 keys, heads 2c and 2c + 1 of each 8
    float z[NT][MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float s0[NT][4] = {}, s1[NT][4] = {};  // even and odd steps: two shorter chains
      const uint8_t* row = st + (16 * t + (lane & 15)) * S::kRow + (lane >> 4) * 16;
#pragma unroll
      for (int k = 0; k < DT; ++k) {
        uint32_t f[4];
        ldmatrix4(f, row + k * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_16816(k & 1 ? s1[n] : s0[n], f, qf[n][k][0], qf[n][k][1]);
      }
      const bool lo = here >> (16 * t + g) & 1, hi = here >> (16 * t + g + 8) & 1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          z[n][t][e] = (e < 2 ? lo : hi) ? (s0[n][e] + s1[n][e]) * a.scale_log2 : -INFINITY;
    }
    float use[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        t0 = fmaxf(t0, fmaxf(z[n][t][0], z[n][t][2]));
        t1 = fmaxf(t1, fmaxf(z[n][t][1], z[n][t][3]));
      }
#pragma unroll
      for (int w = 4; w <= 16; w <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
      }
      t0 = fmaxf(t0, m[n][0]);
      t1 = fmaxf(t1, m[n][1]);
      use[n][0] = t0 == -INFINITY ? 0.f : t0;
      use[n][1] = t1 == -INFINITY ? 0.f : t1;
      if (__any_sync(0xffffffffu, t0 != m[n][0] || t1 != m[n][1])) {
        const float f0 = exp2f(m[n][0] - use[n][0]), f1 = exp2f(m[n][1] - use[n][1]);
        l[n][0] *= f0;
        l[n][1] *= f1;
#pragma unroll
        for (int k = 0; k < DT; ++k) {
          o[n][k][0] *= f0; o[n][k][1] *= f1; o[n][k][2] *= f0; o[n][k][3] *= f1;
        }
        m[n][0] = t0;
        m[n][1] = t1;
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      uint32_t high[NT][2], rest[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float p0 = exp2f(z[n][t][0] - use[n][0]), p1 = exp2f(z[n][t][1] - use[n][1]);
        const float p2 = exp2f(z[n][t][2] - use[n][0]), p3 = exp2f(z[n][t][3] - use[n][1]);
        l[n][0] += p0 + p2;
        l[n][1] += p1 + p3;
        const uint32_t ha = pack_bf16x2(p0, p1), hb = pack_bf16x2(p2, p3);
        const uint32_t ra = pack_bf16x2(p0 - __uint_as_float(ha << 16),
                                        p1 - __uint_as_float(ha & 0xffff0000u));
        const uint32_t rb = pack_bf16x2(p2 - __uint_as_float(hb << 16),
                                        p3 - __uint_as_float(hb & 0xffff0000u));
        high[n][0] = movmatrix(ha);
        high[n][1] = movmatrix(hb);
        rest[n][0] = movmatrix(ra);
        rest[n][1] = movmatrix(rb);
      }
      const uint8_t* row = st + (KK + 16 * t + (lane & 7) + (lane >> 4) * 8) * S::kRow +
                           (lane >> 3 & 1) * 16;
#pragma unroll
      for (int k = 0; k < DT; ++k) {
        uint32_t f[4];
        ldmatrix4_trans(f, row + k * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816(o[n][k], f, high[n][0], high[n][1]);
          mma_16816(o[n][k], f, rest[n][0], rest[n][1]);
        }
      }
    }
  }

  __device__ __forceinline__ void sums(float* ms, float* ls) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], w);
        if (g == 0) {
          ms[8 * n + 2 * c + x] = m[n][x];
          ls[8 * n + 2 * c + x] = l[n][x];
        }
      }
  }
  __device__ __forceinline__ void outputs(float* out) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < DT; ++k) {
        float* p = out + (8 * n + 2 * c) * (D + 4) + 16 * k + g;
        p[0] = o[n][k][0];
        p[D + 4] = o[n][k][1];
        p[8] = o[n][k][2];
        p[D + 12] = o[n][k][3];
      }
  }
};

// A cut run's parts for one head, and where its results go.
template <class S>
struct DecParts {
  static constexpr int D = S::D;
  int n, first, rest;    // parts; slot of the first, then rest + 2 i
  const float* part;
  int64_t row;

  __device__ __forceinline__ DecParts(const DecodeArgs& a, const int4& j, int h) {
    n = 1 + (j.w - (j.z & ~1)) / 2;
    first = j.z;
    rest = j.z & ~1;
    part = a.part + (int64_t)h * (D + 2);
    row = (int64_t)j.x * a.hq + j.y / a.hgroups * a.group + j.y % a.hgroups * S::H + h;
  }
  __device__ __forceinline__ const float* operator[](int i) const {
    return part + (int64_t)(i == 0 ? first : rest + 2 * i) * (S::H * (D + 2));
  }
};
template <class S>
__device__ __forceinline__ int dec_heads_of(const DecodeArgs& a, const int4& j) {
  return min(S::H, a.group - j.y % a.hgroups * S::H);
}

// Joins the parts of runs that were cut; two forms, both for any number of parts.
// Few parts: a block per entry of joins, a warp per head; the first 8 parts' values
// are on their way before the weights are known.
template <class S>
__global__ void __launch_bounds__(32 * S::H) decode_join_few_kernel(const DecodeArgs a) {
  using T = typename S::T;
  constexpr int D = S::D, E2 = D / 64, kBatch = 8;
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  dependency_wait();
  const int4 j = a.joins[blockIdx.x];
  if (j.x < 0 || h >= dec_heads_of<S>(a, j)) return;
  const DecParts<S> p(a, j, h);
  auto values = [&](int i, int e) {  // elements 64 e + 2 lane, + 1
    return *reinterpret_cast<const float2*>(p[i] + 64 * e + 2 * lane);
  };
  float2 v[kBatch][E2];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int e = 0; e < E2; ++e) v[k][e] = i0 + k < p.n ? values(i0 + k, e) : make_float2(0.f, 0.f);
  };
  fetch(0);
  // each lane a part's maximum and sum, 32 at a time
  float mm = -INFINITY, ll = 0.f, acc[2 * E2] = {};
  for (int i0 = 0; i0 < p.n; i0 += 32) {
    const int i = i0 + lane;
    const float m = i < p.n ? p[i][D] : -INFINITY, l = i < p.n ? p[i][D + 1] : 0.f;
    const float m_new = fmaxf(mm, warp_max(m)), mu = m_new == -INFINITY ? 0.f : m_new;
    const float scale = exp2f(mm - mu), f = i < p.n ? exp2f(m - mu) : 0.f;
    mm = m_new;
    ll = ll * scale + warp_sum(l * f);
#pragma unroll
    for (int e = 0; e < 2 * E2; ++e) acc[e] *= scale;
    for (int k0 = 0; k0 < min(32, p.n - i0); k0 += kBatch) {
      if (i0 + k0 > 0) fetch(i0 + k0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k0 + k);  // 0 behind the last part
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          acc[2 * e] = fmaf(v[k][e].x, w, acc[2 * e]);
          acc[2 * e + 1] = fmaf(v[k][e].y, w, acc[2 * e + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2 * E2; ++e)
    static_cast<T*>(a.out)[p.row * D + 64 * (e / 2) + 2 * lane + e % 2] =
        from_f32<T>(ll == 0.f ? 0.f : acc[e] / ll);
  if (a.lse && lane == 0) a.lse[p.row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// Many parts: a block per entry of joins and head, G groups of D threads that take
// every G-th part (65793 keys of one sequence come in 74 parts: 28 us as a chain of
// dependent loads, 3 us so).
constexpr int kJoinThreads = 512;
template <class S>
__global__ void __launch_bounds__(kJoinThreads) decode_join_many_kernel(const DecodeArgs a) {
  using T = typename S::T;
  constexpr int D = S::D;
  constexpr int G = kJoinThreads / D, W = kJoinThreads / 32, kEarly = 16;
  __shared__ float f[kDecMaxBlocks], red[2][W], acc_g[G][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  dependency_wait();
  const int4 j = a.joins[blockIdx.x];
  if (j.x < 0 || h >= dec_heads_of<S>(a, j)) return;
  const DecParts<S> p(a, j, h);
  const int e = tid % D, g = tid / D;
  float early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) early[k] = g + G * k < p.n ? p[g + G * k][e] : 0.f;
  // n <= kDecMaxBlocks <= kJoinThreads: a part's maximum and sum per thread
  static_assert(kDecMaxBlocks <= kJoinThreads, "");
  float m = -INFINITY, l = 0.f;
  if (tid < p.n) {
    m = p[tid][D];
    l = p[tid][D + 1];
  }
  const float wm = warp_max(m);
  if (lane == 0) red[0][warp] = wm;
  __syncthreads();
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) mm = fmaxf(mm, red[0][w]);
  const float mu = mm == -INFINITY ? 0.f : mm;
  if (tid < p.n) {
    f[tid] = exp2f(m - mu);
    l *= f[tid];
  }
  const float wl = warp_sum(l);
  if (lane == 0) red[1][warp] = wl;
  __syncthreads();
  float ll = 0.f, acc = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) ll += red[1][w];
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (g + G * k < p.n) acc = fmaf(early[k], f[g + G * k], acc);
#pragma unroll 4
  for (int i = g + G * kEarly; i < p.n; i += G) acc = fmaf(p[i][e], f[i], acc);
  acc_g[g][e] = acc;
  __syncthreads();
  if (g) return;
#pragma unroll
  for (int i = 1; i < G; ++i) acc += acc_g[i][e];
  static_cast<T*>(a.out)[p.row * D + e] = from_f32<T>(ll == 0.f ? 0.f : acc / ll);
  if (a.lse && tid == 0) a.lse[p.row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

namespace {

struct DecLayout {
  size_t status, joins, part, total;
};
// Query heads of a run: those of a KV head in as few runs as a kernel can hold (bf16 16, fp32
// 8), the runs as even as they can be (100 fp32 sequences of 5000 keys, 12 heads on one KV
// head: 168 us in two runs of 6, 188 in 8 and 4). 144 bf16 sequences of 2987 keys, 12 heads of
// 64 on one KV head, 24 us in one run of 16 and 34 in two of 8; fp32, 4 sequences up to 88849
// keys with 4 heads on each of 2 KV heads, 92 us in a run of 4 and 108 in one of 8 with empty
// heads.
int dec_heads(int group, int dtype) {
  if (dtype == ADASPARK_BF16) return group <= 8 ? 8 : 16;
  const int runs = (group + 7) / 8;
  return std::max(2, (group + runs - 1) / runs);
}

DecLayout dec_layout(int d, int heads) {
  DecLayout L{};
  size_t o = align_up(sizeof(WsHeader));
  L.status = o;
  o = align_up(o + kDecMaxBlocks * sizeof(int32_t));
  L.joins = o;
  o = align_up(o + kDecMaxBlocks * sizeof(int4));
  L.part = o;
  o = align_up(o + (size_t)kDecMaxBlocks * 2 * heads * (d + 2) * sizeof(float));
  L.total = o;
  return L;
}

int64_t dec_run_tiles(int64_t max_len, int tile) { return (max_len + tile - 1) / tile; }

template <class M>
int launch_decode(DecodeArgs a, int sms, cudaStream_t s) {
  using S = typename M::S;
  // no more blocks than tiles the tables can hold
  const int64_t runs = (int64_t)a.n_seqs * a.hkv * a.hgroups;
  const int64_t tiles = runs * dec_run_tiles(a.max_len, S::kTile);
  // Blocks per SM: two, and three where the kernel allows it and blocks walk several runs
  // each: 256 bf16 sequences up to 300 keys, 28 heads on 4, 23 us at three and 25 at two; 61
  // sequences up to 9001 keys, 16 heads on 2, 52 and 49 us. fp32 runs of up to 4 heads
  // always three.
  const int per_sm = sizeof(typename S::T) == 2 && runs <= sms ? 2 : S::kBlocks;
  int64_t grid = per_sm * (int64_t)sms;
  if (grid > kDecMaxBlocks) grid = kDecMaxBlocks;
  if (grid > tiles) grid = tiles;
  a.in_page = a.cs.page_size % S::kKeys == 0;
  a.tile_pages = S::kTile / a.cs.page_size;
  a.tile_rest = S::kTile % a.cs.page_size;
  // Few short runs: a cluster of blocks each, as many as the tables' longest run fills, with
  // up to 2 tiles a block, or 6 where the clusters have more blocks than the GPU SMs (bf16, 28
  // heads on 4, pages of 16; cluster and line: 1 sequence of 1000 keys 6.2 and 6.9 us, of 2040
  // 7.9 and 7.0; 12 of 3000 18.1 and 19.7, 12 of 1 to 3000 14.6 and 15.6; with 8 tiles a block 6
  // of 1 to 4000 13.2 and 11.8).
  const int64_t run_tiles = dec_run_tiles(a.max_len, S::kTile);
  for (int C = kDecCluster; C >= 1; C /= 2) {
    if (run_tiles * 2 <= C || run_tiles > (runs * C > sms ? 6 : 2) * C ||
        runs * C > S::kBlocks * (int64_t)sms || runs * C > kDecMaxBlocks)
      continue;
    const int rc = allow_smem(decode_cluster_kernel<M>, S::kSmem);
    if (rc != ADASPARK_OK) return rc;
    return cuda_status(launch_after("decode_attn", decode_cluster_kernel<M>,
                                    dim3((unsigned)(runs * C)), dim3(kDecWarps * 32), S::kSmem, s,
                                    C, a, C));
  }
  a.by_run = runs <= grid;
  // Two to an SM ask for so much shared memory that a third does not fit: else the blocks of a
  // call that comes up while the last one's join runs pile up on some SMs (61 sequences, back
  // to back: 60 us instead of 56).
  const int smem = per_sm == 2 ? std::max(S::kSmem, 80 << 10) : S::kSmem;
  int rc = allow_smem(decode_kernel<M>, smem);
  if (rc == ADASPARK_OK)
    rc = cuda_status(launch_after("decode_attn", decode_kernel<M>, dim3((unsigned)grid),
                                  dim3(kDecWarps * 32), smem, s, 1, a));
  if (rc != ADASPARK_OK) return rc;
  // Parts per run, about: from some 16 on their loads go side by side in a block (3 sequences of
  // 12000 keys, 25 parts a run, 19.7 us and 20.8 with a warp for all parts of a head; 6 of 8000,
  // 12 parts, 24.9 and 24.1).
  const unsigned entries = (unsigned)(a.by_run ? runs : grid);
  if (grid / runs >= 16)
    return cuda_status(launch_after("decode_join", decode_join_many_kernel<S>,
                                    dim3(entries, a.group < S::H ? a.group : S::H),
                                    dim3(kJoinThreads), 0, s, 1, a));
  return cuda_status(launch_after("decode_join", decode_join_few_kernel<S>, dim3(entries),
                                  dim3(32 * S::H), 0, s, 1, a));
}

template <int H>
int launch_fp32(const DecodeArgs& a, int d, int sms, cudaStream_t s) {
  return d == 128 ? launch_decode<DecFp32<128, H>>(a, sms, s)
                  : launch_decode<DecFp32<64, H>>(a, sms, s);
}

}  // namespace
}  // namespace adaspark

using namespace adaspark;

extern "C" {

size_t adaspark_decode_attn_workspace(int n_seqs, int hq, int hkv, int d, int dtype) {
  if (n_seqs < 1 || n_seqs > kMaxSeqs || !head_sizes_ok(hq, hkv, d, dtype)) return 0;
  return dec_layout(d, dec_heads(hq / hkv, dtype)).total;
}

int adaspark_decode_attn(const void* Q, int64_t q_ts, int64_t q_hs, const void* k_cache,
                         const void* v_cache, int64_t c_ps, int64_t c_ts, int64_t c_hs,
                         int n_pages, int page_size, int dtype, const int32_t* block_table,
                         int64_t table_stride, int max_pages, const int32_t* seq_lens, int n_seqs,
                         int hq, int hkv, int d, float scale, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!Q || !block_table || !seq_lens || !out || !workspace) return ADASPARK_EINVAL;
  if (n_seqs < 1 || n_seqs > kMaxSeqs || max_pages < 1 || !head_sizes_ok(hq, hkv, d, dtype))
    return ADASPARK_EINVAL;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634074);
  if (!std::isfinite(scale_log2)) return ADASPARK_EINVAL;
  const CacheRows cs{c_ps, c_ts, c_hs, n_pages, page_size};
  if (!cache_ok(k_cache, v_cache, cs, hkv, d, dtype)) return ADASPARK_EINVAL;
  if ((int64_t)max_pages * page_size > INT32_MAX - 1024) return ADASPARK_EINVAL;
  const int heads = dec_heads(hq / hkv, dtype), hgroups = (hq / hkv + heads - 1) / heads;
  const int tile = 4096 / (d * (int)elem_size(dtype)) * kDecWarps;
  if ((int64_t)n_seqs * hkv * hgroups * dec_run_tiles((int64_t)max_pages * page_size, tile) >
      INT32_MAX)
    return ADASPARK_EINVAL;
  if (!rows_aligned(Q, q_ts, q_hs, dtype) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return ADASPARK_EINVAL;
  if (!aligned(workspace, kAlign) ||
      workspace_bytes < adaspark_decode_attn_workspace(n_seqs, hq, hkv, d, dtype))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  const DecLayout L = dec_layout(d, heads);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeArgs a{};
  a.hdr = reinterpret_cast<WsHeader*>(ws);
  a.q = Q; a.qs = {q_ts, q_hs};
  a.kc = k_cache; a.vc = v_cache; a.cs = cs;
  a.table = block_table; a.table_stride = table_stride; a.lens = seq_lens;
  a.out = out; a.lse = lse;
  a.scale_log2 = scale_log2;
  a.n_seqs = n_seqs; a.max_len = max_pages * page_size;
  a.hq = hq; a.hkv = hkv; a.group = hq / hkv;
  a.hgroups = hgroups;
  a.status = reinterpret_cast<int32_t*>(ws + L.status);
  a.joins = reinterpret_cast<int4*>(ws + L.joins);
  a.part = reinterpret_cast<float*>(ws + L.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == ADASPARK_BF16) {
    if (heads == 8)
      return d == 128 ? launch_decode<DecBf16<128, 1>>(a, sms, s)
                      : launch_decode<DecBf16<64, 1>>(a, sms, s);
    return d == 128 ? launch_decode<DecBf16<128, 2>>(a, sms, s)
                    : launch_decode<DecBf16<64, 2>>(a, sms, s);
  }
  switch (heads) {
    case 2: return launch_fp32<2>(a, d, sms, s);
    case 3: return launch_fp32<3>(a, d, sms, s);
    case 4: return launch_fp32<4>(a, d, sms, s);
    case 5: return launch_fp32<5>(a, d, sms, s);
    case 6: return launch_fp32<6>(a, d, sms, s);
    case 7: return launch_fp32<7>(a, d, sms, s);
    default: return launch_fp32<8>(a, d, sms, s);
  }
}

}  // extern "C"
