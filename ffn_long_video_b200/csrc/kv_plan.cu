// The page plan of a paged key-value cache: sequences go from their old to
// their new lengths, pages move between the block tables and the free list, and
// every new token gets its slot (page * page_size + offset) and its position.
//
// With P(n) = ceil(n / page_size), sequence i takes max(P(new) - P(old), 0)
// pages or gives back max(P(old) - P(new), 0). Pages given back are pushed onto
// the free list so that the t-th page taken (sequences ascending, then pages
// ascending) is the t-th page given back while there are any, then the list's
// last one, and so on downwards: a step from new to old lengths undoes the step
// from old to new, free list included. A plan that cannot be carried out
// changes nothing.
//
// Latency-bound: a block sums the sequences' takes, gifts and new tokens and writes
// slots, table and list entries. A step's few rows take one block; many rows
// (prompts) the whole GPU, where every block sums for itself, nobody reads what
// another block writes, and the free count, which all of them read, follows in a
// second kernel. Sequences that are too many for that are summed by a kernel ahead.
#include <algorithm>

#include "serve.h"

namespace adaspark {

struct PlanArgs {
  WsHeader* hdr;
  const int32_t *old_lens, *new_lens;
  int32_t* table;
  int64_t table_stride;
  int32_t *free_pages, *n_free;
  int32_t *starts, *slots, *positions;
  int32_t* status;               // workspace: status bits of each block
  int32_t *take0, *give0;        // workspace: pages taken / given by earlier sequences
  int32_t n_seqs, max_pages, page_size, n_pages, n_rows;
  int32_t chunk;                 // rows a warp takes at a time
  int32_t blocks;                // blocks that write status words (0: the header holds all)
  uint32_t div_mul, div_shift;   // n / page_size = n * div_mul >> div_shift for 0 <= n < 2^31
};

// Totals of a plan; the workspace header keeps them for the second kernel.
struct PlanTotals {
  int32_t ok, rows, take, give, n_free;
};
__device__ __forceinline__ PlanTotals* plan_totals(WsHeader* h) {
  return reinterpret_cast<PlanTotals*>(h->stats);
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 1024;      // sequences whose sums are kept in shared memory
// Up to here one block writes a plan's rows, 4 each thread. Plans one after another, one
// block and all: 64 sequences that gain 161 tokens 3.0 and 4.5 us, 250 that gain 4000 5.6 and
// 6.3, 8000 6.6 and 5.6. 300 sequences, a third of them gone and a third new with 825
// thousand tokens: 7.8 us (7 MB of slots, positions and page numbers: 1 us at 6.46 TB/s; the
// rest is one launch, three dependent reads and the second launch), 10.2 with the sums in a
// kernel of their own.
constexpr int kPlanOneBlock = 4096;

// Per-sequence values that the writes search, in shared memory or (more than
// kPlanSeqs sequences) in global memory.
struct PlanSums {
  const int32_t *old_lens, *new_lens, *take0, *give0, *starts;
};
struct PlanShared {
  int32_t old_lens[kPlanSeqs], new_lens[kPlanSeqs], take0[kPlanSeqs], give0[kPlanSeqs],
      starts[kPlanSeqs];
};

__device__ __forceinline__ int plan_div(const PlanArgs& a, int n) {
  return (int)((uint64_t)(uint32_t)n * a.div_mul >> a.div_shift);
}
// Pages of n tokens.
__device__ __forceinline__ int plan_pages(const PlanArgs& a, int n) {
  const int q = plan_div(a, n);
  return q + (n != q * a.page_size);
}

// Inclusive sums of three values over the warp.
template <typename I>
__device__ __forceinline__ void warp_scan3(I (&v)[3]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const I u = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += u;
    }
  }
}

// Sums over the sequences (a block of whole warps), the plan's check, its totals;
// block 0 writes starts and status and, with COUNT, n_free. KEEP: the sums stay in
// shared memory (n_seqs <= kPlanSeqs), else they go to the workspace.
constexpr int kPlanTooMuch = 1 << 21;  // 1024 values below it sum up in 31 bits
template <bool KEEP, bool COUNT>
__device__ __forceinline__ PlanTotals plan_sums(const PlanArgs& a, PlanShared* sh) {
  __shared__ int warp_sum[2][kPlanThreads / 32][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool first = blockIdx.x == 0;
  const long long F = *a.n_free;
  const long long most = (long long)a.max_pages * a.page_size;
  long long carry[3] = {0, 0, 0};
  bool bad = false;
  for (int base = 0, buf = 0; base < a.n_seqs; base += blockDim.x, buf ^= 1) {
    const int i = base + threadIdx.x;
    int o = 0, n = 0;
    if (i < a.n_seqs) {
      o = a.old_lens[i];
      n = a.new_lens[i];
      if (KEEP) {
        sh->old_lens[i] = o;
        sh->new_lens[i] = n;
      }
    }
    const bool wrong = o < 0 || n < 0 || o > most || n > most;
    if (wrong) o = n = 0;
    const int po = plan_pages(a, o), pn = plan_pages(a, n);
    const int own[3] = {max(pn - po, 0), max(po - pn, 0), max(n - o, 0)};
    // sums of this round in 32 bits where they fit, which one barrier tells; else in 64
    const bool large = max(max(own[0], own[1]), own[2]) >= kPlanTooMuch;
    bad |= wrong;
    long long before[3], total[3];
    if (!__syncthreads_or(large)) {
      int v[3] = {own[0], own[1], own[2]};
      warp_scan3(v);
      if (lane == 31) {
#pragma unroll
        for (int k = 0; k < 3; ++k) warp_sum[buf][warp][k] = v[k];
      }
      __syncthreads();
      // every warp sums the warps' totals
      int w[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k] = lane < warps ? warp_sum[buf][lane][k] : 0;
      warp_scan3(w);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int up = __shfl_sync(0xffffffffu, w[k], max(warp - 1, 0));
        before[k] = v[k] - own[k] + (warp ? up : 0);
        total[k] = __shfl_sync(0xffffffffu, w[k], 31);
      }
    } else {
      __shared__ long long wide[kPlanThreads / 32][3];
      long long v[3] = {own[0], own[1], own[2]};
      warp_scan3(v);
      __syncthreads();
      if (lane == 31) {
#pragma unroll
        for (int k = 0; k < 3; ++k) wide[warp][k] = v[k];
      }
      __syncthreads();
      long long w[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k] = lane < warps ? wide[lane][k] : 0;
      warp_scan3(w);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long up = __shfl_sync(0xffffffffu, w[k], max(warp - 1, 0));
        before[k] = v[k] - own[k] + (warp ? up : 0);
        total[k] = __shfl_sync(0xffffffffu, w[k], 31);
      }
    }
    if (i < a.n_seqs) {
      // sums of a plan that holds fit 31 bits; another's are not used
      (KEEP ? sh->take0 : a.take0)[i] = (int32_t)(carry[0] + before[0]);
      (KEEP ? sh->give0 : a.give0)[i] = (int32_t)(carry[1] + before[1]);
      if (KEEP) sh->starts[i] = (int32_t)(carry[2] + before[2]);
      if (first) a.starts[i] = (int32_t)(carry[2] + before[2]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) carry[k] += total[k];
  }
  // n_free was read, the sums are there
  const bool any_bad = __syncthreads_or(bad);
  const long long left = F + carry[1] - carry[0];
  // lengths the tables hold, rows for every new token, no more pages than there are
  const bool sound = !any_bad && carry[2] <= a.n_rows && F >= 0 && F <= a.n_pages &&
                     carry[1] <= a.n_pages && left <= a.n_pages;
  const bool ok = sound && left >= 0;
  if (!ok && first)
    for (int i = threadIdx.x; i < a.n_seqs; i += blockDim.x) a.starts[i] = 0;
  const PlanTotals t{ok, (int32_t)carry[2], (int32_t)carry[0], (int32_t)carry[1], (int32_t)F};
  if (first && threadIdx.x == 0) {
    a.starts[a.n_seqs] = ok ? t.rows : 0;
    if (COUNT && ok) *a.n_free = (int32_t)left;
    a.hdr->status = ok ? 0u : sound ? ADASPARK_DEV_PAGES : ADASPARK_DEV_BAD_LAYOUT;
    a.hdr->detail = ok ? 0u : ADASPARK_PLAN_REFUSED;
    a.hdr->n_block_status = a.blocks;
  }
  return t;
}

// Index of the last entry of first[0..n) that is <= x (first is nondecreasing, first[0] = 0):
// the sequence that x belongs to.
__device__ __forceinline__ int plan_find(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The same for one x of a whole warp, 32 entries a step.
__device__ __forceinline__ int plan_find_warp(const int32_t* first, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32, i = lane * step;
    const uint32_t at_most = __ballot_sync(0xffffffffu, i < len && first[lo + min(i, len - 1)] <= x);
    const int skip = max(__popc(at_most) - 1, 0) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  return lo;
}

// The g-th page given back: from its sequence's table row, which this plan does not write
// there. `s`: a sequence no later than the one it belongs to.
__device__ __forceinline__ int plan_given(const PlanArgs& a, const PlanSums& p, int g, int s) {
  while (s + 1 < a.n_seqs && p.give0[s + 1] <= g) ++s;
  const int col = plan_pages(a, p.new_lens[s]) + g - p.give0[s];
  return a.table[s * a.table_stride + col];
}

// The i-th page taken. List entries from n_free on are written by this plan, those below are not.
__device__ __forceinline__ int plan_taken(const PlanArgs& a, const PlanSums& p,
                                          const PlanTotals& t, int i, int s) {
  return i < t.give ? plan_given(a, p, i, s) : a.free_pages[t.n_free - 1 - (i - t.give)];
}

__device__ __forceinline__ void plan_row(const PlanArgs& a, int r, int pos, int page, int in_page,
                                         bool* bad) {
  int slot = -1;
  if (page >= 0 && page < a.n_pages)
    slot = page * a.page_size + in_page;
  else
    *bad = true;
  a.slots[r] = slot;
  a.positions[r] = pos;
}

// Slots, positions, table and list entries, by `warps` warps of which this is
// `warp`. A page that is taken is written to its table by whoever has its first
// token, which is always a new one. Returns whether this thread met a page number
// that the pool does not have, for a new token or among the pages given back (which
// go onto the list as they are, so that the plan can be undone).
__device__ __forceinline__ bool plan_write(const PlanArgs& a, const PlanSums& p,
                                           const PlanTotals& t, int warp, int warps) {
  const int lane = threadIdx.x & 31, rows = t.ok ? t.rows : 0;
  bool bad = false;
  for (int r0 = warp * a.chunk; r0 < a.n_rows; r0 += warps * a.chunk) {
    const int r1 = min(r0 + a.chunk, a.n_rows), r2 = min(r1, rows);
    for (int r = max(r0, rows) + lane; r < r1; r += 32) {
      a.slots[r] = -1;
      a.positions[r] = 0;
    }
    if (r0 >= r2) continue;
    int s = plan_find_warp(p.starts, a.n_seqs, r0);
    const int span = plan_find_warp(p.starts, a.n_seqs, r2 - 1) + 1 - s;
    if (span <= 8) {
      // few sequences: the warp looks up 32 pages of one at a time
      for (int ra = r0; ra < r2; ++s) {
        const int st = p.starts[s], rb = s + 1 < a.n_seqs ? min(r2, p.starts[s + 1]) : r2;
        const int o = p.old_lens[s], shift = o - st;  // position of row r: r + shift
        const int held = plan_pages(a, o);
        const int last = ra < rb ? plan_div(a, rb - 1 + shift) : -1;
        for (int c0 = ra < rb ? plan_div(a, ra + shift) : 0; c0 <= last; c0 += 32) {
          const int col = c0 + lane, taken = p.take0[s] - held;  // column c takes page taken + c
          const int from = taken + max(c0, held);
          const int giver = c0 + 31 >= held && from < t.give
                                ? plan_find_warp(p.give0, a.n_seqs, from)
                                : 0;
          int page = -1;
          if (col <= last && col < held) {
            page = a.table[s * a.table_stride + col];
          } else if (col <= last) {
            page = plan_taken(a, p, t, taken + col, giver);
            if (col * a.page_size - shift >= ra) a.table[s * a.table_stride + col] = page;
          }
          // rows of these pages; 64 bits: the last page's end may pass 2^31
          const int rc = (int)min((long long)rb, (long long)(c0 + 32) * a.page_size - shift);
          for (; ra < rc; ra += 32) {
            const int r = min(ra + lane, rc - 1), pos = r + shift, c = plan_div(a, pos);
            const int pg = __shfl_sync(0xffffffffu, page, c - c0);
            if (ra + lane < rc) plan_row(a, r, pos, pg, pos - c * a.page_size, &bad);
          }
          ra = rc;
        }
      }
    } else {
      // many sequences: a lane looks up its own row
      const int s0 = s;
      for (int r = r0 + lane; r < r2; r += 32) {
        s = s0 + plan_find(p.starts + s0, span, r);
        const int o = p.old_lens[s], pos = o + r - p.starts[s], col = plan_div(a, pos);
        const int held = plan_pages(a, o), i = p.take0[s] + col - held;
        int page;
        if (col < held) {
          page = a.table[s * a.table_stride + col];
        } else {
          page = plan_taken(a, p, t, i, i < t.give ? plan_find(p.give0, a.n_seqs, i) : 0);
          if (col * a.page_size == pos) a.table[s * a.table_stride + col] = page;
        }
        plan_row(a, r, pos, page, pos - col * a.page_size, &bad);
      }
    }
  }
  if (!t.ok) return bad;
  for (int g = t.take + warp * 32 + lane; g < t.give; g += warps * 32) {
    const int page = plan_given(a, p, g, plan_find(p.give0, a.n_seqs, g));
    bad |= page < 0 || page >= a.n_pages;
    a.free_pages[t.n_free + t.give - 1 - g] = page;
  }
  return bad;
}

__device__ __forceinline__ PlanSums plan_kept(const PlanShared& sh) {
  return {sh.old_lens, sh.new_lens, sh.take0, sh.give0, sh.starts};
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ PlanShared sh;
  dependency_wait();
  const PlanTotals t = plan_sums<true, true>(a, &sh);
  __syncthreads();
  const bool bad = plan_write(a, plan_kept(sh), t, threadIdx.x >> 5, blockDim.x >> 5);
  if (__syncthreads_or(bad) && threadIdx.x == 0) {
    a.hdr->status = ADASPARK_DEV_BAD_LAYOUT;
    a.hdr->detail = 0x8200u;
  }
}

__device__ __forceinline__ void plan_block_status(const PlanArgs& a, bool bad) {
  const bool any = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.status[blockIdx.x] = any ? ADASPARK_DEV_BAD_LAYOUT : 0;
}

// Many rows, up to kPlanSeqs sequences; n_free is written by plan_count_kernel. One block an
// SM: 7.8 us for the 825 thousand tokens above, 8.1 with two of half the size, 9.2 with four.
__global__ void __launch_bounds__(kPlanThreads) plan_wide_kernel(const PlanArgs a) {
  __shared__ PlanShared sh;
  dependency_wait();
  const PlanTotals t = plan_sums<true, false>(a, &sh);
  if (blockIdx.x == 0 && threadIdx.x == 0) *plan_totals(a.hdr) = t;
  __syncthreads();
  constexpr int W = kPlanThreads / 32;
  plan_block_status(a, plan_write(a, plan_kept(sh), t, blockIdx.x * W + (threadIdx.x >> 5),
                                  gridDim.x * W));
}
__global__ void plan_count_kernel(const PlanArgs a) {
  dependency_wait();
  const PlanTotals t = *plan_totals(a.hdr);
  if (t.ok) *a.n_free = t.n_free + t.give - t.take;
}

// More sequences: their sums in the workspace (2000 that gain 8000 tokens: 13.8 us).
__global__ void __launch_bounds__(kPlanThreads) plan_sums_kernel(const PlanArgs a) {
  dependency_wait();
  const PlanTotals t = plan_sums<false, true>(a, nullptr);
  if (threadIdx.x == 0) *plan_totals(a.hdr) = t;
}
__global__ void __launch_bounds__(kPlanThreads) plan_write_kernel(const PlanArgs a) {
  dependency_wait();
  constexpr int W = kPlanThreads / 32;
  plan_block_status(a, plan_write(a, {a.old_lens, a.new_lens, a.take0, a.give0, a.starts},
                                  *plan_totals(a.hdr), blockIdx.x * W + (threadIdx.x >> 5),
                                  gridDim.x * W));
}

constexpr int kPlanMaxBlocks = 1024;

}  // namespace adaspark

using namespace adaspark;

extern "C" {

size_t adaspark_kv_plan_workspace(int n_seqs) {
  if (n_seqs < 1 || n_seqs > kMaxSeqs) return 0;
  return align_up(sizeof(WsHeader)) + align_up(kPlanMaxBlocks * sizeof(int32_t)) +
         2 * align_up((size_t)n_seqs * sizeof(int32_t));
}

int adaspark_kv_plan(const int32_t* old_lens, const int32_t* new_lens, int n_seqs, int page_size,
                     int32_t* block_table, int64_t table_stride, int max_pages,
                     int32_t* free_pages, int n_pages, int32_t* n_free, int32_t* token_starts,
                     int32_t* slots, int32_t* positions, int n_rows, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!old_lens || !new_lens || !block_table || !free_pages || !n_free || !token_starts || !slots ||
      !positions || !workspace)
    return ADASPARK_EINVAL;
  if (n_seqs < 1 || page_size < 1 || max_pages < 1 || n_pages < 1 || n_rows < 1)
    return ADASPARK_EINVAL;
  if (table_stride < max_pages && n_seqs > 1) return ADASPARK_EINVAL;
  if ((int64_t)n_pages * page_size > INT32_MAX) return ADASPARK_EINVAL;
  // room for the kernels' strides in 32 bits
  if (n_seqs > kMaxSeqs || n_pages > (1 << 30) || n_rows > (1 << 30)) return ADASPARK_EINVAL;
  for (const void* p : {(const void*)old_lens, (const void*)new_lens, (const void*)block_table,
                        (const void*)free_pages, (const void*)n_free, (const void*)token_starts,
                        (const void*)slots, (const void*)positions})
    if (!aligned(p, 4)) return ADASPARK_EINVAL;
  if (!aligned(workspace, kAlign) || workspace_bytes < adaspark_kv_plan_workspace(n_seqs))
    return ADASPARK_EINVAL;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != ADASPARK_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PlanArgs a{};
  a.hdr = reinterpret_cast<WsHeader*>(ws);
  a.status = reinterpret_cast<int32_t*>(ws + align_up(sizeof(WsHeader)));
  a.take0 = a.status + align_up(kPlanMaxBlocks * sizeof(int32_t)) / sizeof(int32_t);
  a.give0 = a.take0 + align_up((size_t)n_seqs * sizeof(int32_t)) / sizeof(int32_t);
  a.old_lens = old_lens; a.new_lens = new_lens;
  a.table = block_table; a.table_stride = table_stride;
  a.free_pages = free_pages; a.n_free = n_free;
  a.starts = token_starts; a.slots = slots; a.positions = positions;
  a.n_seqs = n_seqs; a.max_pages = max_pages; a.page_size = page_size;
  a.n_pages = n_pages; a.n_rows = n_rows;
  // with 2^(k-1) < page_size <= 2^k, ceil(2^(31+k) / page_size) < 2^32 divides every n < 2^31
  int k = 0;
  while ((int64_t)1 << k < page_size) ++k;
  a.div_shift = 31 + k;
  a.div_mul = (uint32_t)((((uint64_t)1 << (31 + k)) + page_size - 1) / page_size);
  if (n_rows <= kPlanOneBlock && n_seqs <= kPlanSeqs) {
    // no more warps than sequences and rows give work
    const int threads = std::min(kPlanThreads, (std::max(n_seqs, n_rows) + 127) / 128 * 128);
    a.chunk = (n_rows + threads - 1) / threads * 32;
    return cuda_status(launch_after("kv_plan", plan_kernel, dim3(1), dim3(threads), 0, s, 1, a));
  }
  // blocks that fill the GPU until each warp has 512 rows (it has to find its first one)
  constexpr int W = kPlanThreads / 32;
  const bool wide = n_seqs <= kPlanSeqs;
  const int64_t most = sms;
  const int64_t share = (n_rows + most * W * 32 - 1) / (most * W * 32);
  a.chunk = (int)std::min<int64_t>(share, 16) * 32;
  const int64_t want = ((int64_t)n_rows + a.chunk * W - 1) / (a.chunk * W);
  a.blocks = (int)std::min({want, wide ? most : 4 * most, (int64_t)kPlanMaxBlocks});
  const dim3 grid(a.blocks), block(kPlanThreads);
  cudaError_t e;
  if (wide) {
    e = launch_after("kv_plan", plan_wide_kernel, grid, block, 0, s, 1, a);
    if (e == cudaSuccess)
      e = launch_after("kv_plan_count", plan_count_kernel, dim3(1), dim3(1), 0, s, 1, a);
  } else {
    e = launch_after("kv_plan_sums", plan_sums_kernel, dim3(1), dim3(kPlanThreads), 0, s, 1, a);
    if (e == cudaSuccess)
      e = launch_after("kv_plan_write", plan_write_kernel, grid, block, 0, s, 1, a);
  }
  return cuda_status(e);
}

}  // extern "C"
