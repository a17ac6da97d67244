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
// Latency-bound: a first kernel of one block sums the sequences' takes, gifts
// and new tokens; a second writes slots, table entries and list entries.
#include "serve.h"

namespace adaspark {

struct PlanArgs {
  WsHeader* hdr;
  const int32_t *old_lens, *new_lens;
  int32_t* table;
  int64_t table_stride;
  int32_t *free_pages, *n_free;
  int32_t *starts, *slots, *positions;
  int32_t *take0, *give0;        // workspace: pages taken / given by earlier sequences
  int32_t n_seqs, max_pages, page_size, n_pages, n_rows;
};

// Totals of a plan, kept in the workspace header for the second kernel.
struct PlanTotals {
  int32_t ok, rows, take, give, n_free;
};
__device__ __forceinline__ PlanTotals* plan_totals(WsHeader* h) {
  return reinterpret_cast<PlanTotals*>(h->stats);
}

constexpr int kPlanThreads = 1024;

// Inclusive sums of three values over the block, and the block's totals.
__device__ __forceinline__ void block_scan3(long long (&v)[3], long long (&total)[3],
                                            long long (*warp_sum)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const long long u = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += u;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 3; ++k) warp_sum[warp][k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const long long x = warp_sum[w][k];
      if (w < warp) before += x;
      all += x;
    }
    v[k] += before;
    total[k] = all;
  }
  __syncthreads();
}

__device__ __forceinline__ int plan_pages(int n, int page_size) {
  return n / page_size + (n % page_size != 0);
}

__global__ void __launch_bounds__(kPlanThreads) plan_sums_kernel(const PlanArgs a) {
  __shared__ long long warp_sum[kPlanThreads / 32][3];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const long long most = (long long)a.max_pages * a.page_size;
  long long carry[3] = {0, 0, 0};
  for (int base = 0; base < a.n_seqs; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    long long own[3] = {0, 0, 0}, v[3], total[3];
    if (i < a.n_seqs) {
      const int o = a.old_lens[i], n = a.new_lens[i];
      if (o < 0 || n < 0 || o > most || n > most) {
        bad = 1;
      } else {
        const int po = plan_pages(o, a.page_size), pn = plan_pages(n, a.page_size);
        own[0] = max(pn - po, 0);
        own[1] = max(po - pn, 0);
        own[2] = max(n - o, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = own[k];
    block_scan3(v, total, warp_sum);
    if (i < a.n_seqs) {
      // sums of a plan that holds fit 31 bits; another's are not used
      a.take0[i] = (int32_t)(carry[0] + v[0] - own[0]);
      a.give0[i] = (int32_t)(carry[1] + v[1] - own[1]);
      a.starts[i] = (int32_t)(carry[2] + v[2] - own[2]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) carry[k] += total[k];
  }
  __syncthreads();
  const long long F = *a.n_free, left = F + carry[1] - carry[0];
  // lengths the tables hold, rows for every new token, no more pages than there are
  const bool sound = !bad && carry[2] <= a.n_rows && F >= 0 && F <= a.n_pages &&
                     carry[1] <= a.n_pages && left <= a.n_pages;
  const bool ok = sound && left >= 0;
  __syncthreads();  // every thread has read n_free
  if (!ok)
    for (int i = threadIdx.x; i < a.n_seqs; i += kPlanThreads) a.starts[i] = 0;
  if (threadIdx.x == 0) {
    a.starts[a.n_seqs] = ok ? (int32_t)carry[2] : 0;
    PlanTotals* t = plan_totals(a.hdr);
    t->ok = ok;
    t->rows = (int32_t)carry[2];
    t->take = (int32_t)carry[0];
    t->give = (int32_t)carry[1];
    t->n_free = (int32_t)F;
    if (ok) *a.n_free = (int32_t)left;
    a.hdr->status = ok ? 0u : sound ? ADASPARK_DEV_PAGES : ADASPARK_DEV_BAD_LAYOUT;
    a.hdr->detail = ok ? 0u : 0x8100u;
  }
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

// The g-th page given back: from its sequence's table row, which this plan does not write there.
__device__ __forceinline__ int plan_given(const PlanArgs& a, int g) {
  const int s = plan_find(a.give0, a.n_seqs, g);
  const int col = plan_pages(a.new_lens[s], a.page_size) + g - a.give0[s];
  return a.table[s * a.table_stride + col];
}

// The t-th page taken. List entries from n_free on are written by this plan, those below are not.
__device__ __forceinline__ int plan_taken(const PlanArgs& a, const PlanTotals& p, int t) {
  return t < p.give ? plan_given(a, t) : a.free_pages[p.n_free - 1 - (t - p.give)];
}

__global__ void __launch_bounds__(256) plan_write_kernel(const PlanArgs a) {
  const PlanTotals p = *plan_totals(a.hdr);
  const int tid = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
  const int rows = p.ok ? p.rows : 0;
  for (int r = tid; r < a.n_rows; r += step) {
    int slot = -1, pos = 0;
    if (r < rows) {
      const int s = plan_find(a.starts, a.n_seqs, r);
      const int o = a.old_lens[s];
      pos = o + r - a.starts[s];
      const int col = pos / a.page_size, held = plan_pages(o, a.page_size);
      const int page = col < held ? a.table[s * a.table_stride + col]
                                  : plan_taken(a, p, a.take0[s] + col - held);
      if (page >= 0 && page < a.n_pages)
        slot = page * a.page_size + pos % a.page_size;
      else
        set_status(a.hdr, ADASPARK_DEV_BAD_LAYOUT, 0x8200u);
    }
    a.slots[r] = slot;
    a.positions[r] = pos;
  }
  if (!p.ok) return;
  for (int t = tid; t < p.take; t += step) {
    const int s = plan_find(a.take0, a.n_seqs, t);
    const int col = plan_pages(a.old_lens[s], a.page_size) + t - a.take0[s];
    a.table[s * a.table_stride + col] = plan_taken(a, p, t);
  }
  for (int g = p.take + tid; g < p.give; g += step)
    a.free_pages[p.n_free + p.give - 1 - g] = plan_given(a, g);
}

}  // namespace adaspark

using namespace adaspark;

extern "C" {

size_t adaspark_kv_plan_workspace(int n_seqs) {
  if (n_seqs < 1) return 0;
  return align_up(sizeof(WsHeader)) + 2 * align_up((size_t)n_seqs * sizeof(int32_t));
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
  a.take0 = reinterpret_cast<int32_t*>(ws + align_up(sizeof(WsHeader)));
  a.give0 = a.take0 + align_up((size_t)n_seqs * sizeof(int32_t)) / sizeof(int32_t);
  a.old_lens = old_lens; a.new_lens = new_lens;
  a.table = block_table; a.table_stride = table_stride;
  a.free_pages = free_pages; a.n_free = n_free;
  a.starts = token_starts; a.slots = slots; a.positions = positions;
  a.n_seqs = n_seqs; a.max_pages = max_pages; a.page_size = page_size;
  a.n_pages = n_pages; a.n_rows = n_rows;
  cudaError_t e = launch("kv_plan_sums", plan_sums_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e == cudaSuccess) {
    const int64_t want = ((int64_t)n_rows + 255) / 256;
    const unsigned grid = (unsigned)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8);
    e = launch("kv_plan_write", plan_write_kernel, dim3(grid), dim3(256), 0, s, a);
  }
  return cuda_status(e);
}

}  // extern "C"
