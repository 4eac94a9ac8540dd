// Pages of a key/value cache: new tokens written into them, pages copied, sequences forked,
// grown, cut and freed, and the pool compacted (sal_cache_* in sal.h).
//
// The page tables are the only state: a page is in use when one of the first
// ceil(length / page_size) entries of a row names it. resize and compact rebuild that set as
// a bitmap in shared memory (524,288 pages are 64 KB) from the tables they were given, so
// nothing can drift out of step with the tables and freeing is nothing but a shorter length.
// Both run as one block: the bitmap, the scan over the list and the selection of the
// lowest-numbered free pages are a few thousand steps each, and their results (which page
// goes where) are the same whatever the order of the atomics that set the bits. What they
// want copied they leave as (from, to) pairs in the workspace for the copy kernel behind
// them on the stream, which moves the bytes with the whole GPU.
//
// Bound by latency where little moves: eight streams continued by four hypotheses each (a fork, a
// resize of 32 rows and the copies of their last pages, three launches, two of them dependent on
// the one before) take 14.6 us for 1.6 us of bytes. Bound by memory where much does: half of 96 streams of
// a 32-layer cache end and the rest move together, 1.5 GB read and written, in 271 us, 85 % of a plain
// copy's rate (a thread keeps four 16-byte vectors in flight). Up to 749 new positions of ten heads of
// 16 sequences are written in 14.4 us, 80 % of that rate.
#define SAL_CK_FILE 8
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "sal_internal.h"
#include "sal_ptx.cuh"

namespace sal {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kForkInts = 32768;  // shared-memory ints of a fork block's tile: one column of the longest list

struct TableArgs {
  const int32_t *table, *lengths;
  int32_t *table_out, *lengths_out;
  uint32_t* status;
  int sequences, max_pages, pages, page_shift;
};

struct PlanArgs {
  TableArgs t;
  const int32_t *seqs, *new_lengths;  // resize
  int n;
  int left, sinks;  // resize: left < 0 keeps every page
  int32_t* count;   // workspace: pairs to copy
  int2* pairs;      // [pages] (from, to)
  int32_t* freed;   // [pages] free pages in ascending order
  int32_t* offs;    // [sequences] first free page of each list entry
};

struct Layout {
  size_t pairs, freed, offs, bytes;
};
Layout ws_layout(int pages, int sequences) {
  Layout l{};
  l.pairs = 256;
  l.freed = l.pairs + static_cast<size_t>(pages) * 8;
  l.offs = l.freed + static_cast<size_t>(pages) * 4;
  l.bytes = (l.offs + static_cast<size_t>(sequences) * 4 + 255) & ~size_t(255);
  return l;
}

__device__ __forceinline__ int pages_of(int positions, int shift) { return (positions + (1 << shift) - 1) >> shift; }

// Exclusive prefix sum over the block's threads (all of them call it); `total` receives the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sums[lane];
    int z = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, d);
      if (lane >= d) z += y;
    }
    warp_sums[lane] = z - w;
    if (lane == 31) warp_sums[32] = z;
  }
  __syncthreads();
  const int r = warp_sums[warp] + x - v;
  total = warp_sums[32];
  __syncthreads();
  return r;
}

__device__ __forceinline__ int length_of(const TableArgs& t, int seq) {
  return min(max(*SAL_CK_LD(t.lengths + seq, 4), 0), t.max_pages << t.page_shift);
}

// Copies row `seq` and its length to the outputs (nothing to do in place). One warp.
__device__ __forceinline__ void pass_row(const TableArgs& t, int seq) {
  const int lane = threadIdx.x & 31;
  if (t.table_out != t.table) {
    const int64_t at = static_cast<int64_t>(seq) * t.max_pages;
    for (int c = lane; c < t.max_pages; c += 32) *SAL_CK_ST(t.table_out + at + c, 4) = *SAL_CK_LD(t.table + at + c, 4);
  }
  if (lane == 0 && t.lengths_out != t.lengths) *SAL_CK_ST(t.lengths_out + seq, 4) = *SAL_CK_LD(t.lengths + seq, 4);
}

// A list entry of resize: what stays of its sequence and what it asks for.
struct Entry {
  int seq, kept, len;      // positions that stay, new length
  int evict_lo, evict_hi;  // table entries [lo, hi) that are let go
};
__device__ __forceinline__ Entry entry_of(const PlanArgs& a, int i) {
  Entry e;
  e.seq = *SAL_CK_LD(a.seqs + i, 4);
  e.len = *SAL_CK_LD(a.new_lengths + i, 4);
  e.kept = min(length_of(a.t, e.seq), e.len);
  e.evict_lo = e.evict_hi = 0;
  if (a.left >= 0) {
    e.evict_lo = pages_of(a.sinks, a.t.page_shift);
    e.evict_hi = max(0, e.kept - a.left) >> a.t.page_shift;
  }
  return e;
}

// The page in table entry c of an entry's row after the cut, or -1.
__device__ __forceinline__ int kept_page(const PlanArgs& a, const Entry& e, int c) {
  if (c >= e.evict_lo && c < e.evict_hi) return -1;
  const int p = *SAL_CK_LD(a.t.table + static_cast<int64_t>(e.seq) * a.t.max_pages + c, 4);
  return p >= 0 && p < a.t.pages ? p : -1;
}

// Whether the entry grows from inside a page that has been let go. The page's lost positions are
// invisible because its entry names no page: with a page for the new ones they would be visible again
// and hold whatever it held last.
__device__ __forceinline__ bool grows_from_lost(const PlanArgs& a, const Entry& e) {
  return e.len > e.kept && (e.kept & ((1 << a.t.page_shift) - 1)) && kept_page(a, e, e.kept >> a.t.page_shift) < 0;
}

// Whether the entry's partly filled last page (it is there) is shared, so that it has to be replaced by
// a copy of itself, page `from`, before it grows.
__device__ __forceinline__ bool replaces(const PlanArgs& a, const Entry& e, const uint32_t* multi, int& from) {
  from = -1;
  if (e.len <= e.kept || !(e.kept & ((1 << a.t.page_shift) - 1))) return false;
  const int p = kept_page(a, e, e.kept >> a.t.page_shift);
  if (p < 0 || !((multi[p >> 5] >> (p & 31)) & 1u)) return false;
  from = p;
  return true;
}

__global__ void __launch_bounds__(kPlanThreads, 1) resize_kernel(const PlanArgs a) {
  extern __shared__ uint32_t sm[];
  const TableArgs& t = a.t;
  const int words = (t.pages + 31) >> 5, seq_words = (t.sequences + 31) >> 5;
  uint32_t* used = sm;              // pages that some row names after the cuts
  uint32_t* multi = sm + words;     // ... that more than one names
  uint32_t* listed = multi + words;  // sequences on the list
  __shared__ int warp_sums[33];
  __shared__ int bad, lost, n_pairs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < 2 * words + seq_words; i += kPlanThreads) sm[i] = 0;
  if (tid == 0) bad = lost = n_pairs = 0;
  __syncthreads();
  const int capacity = t.max_pages << t.page_shift;
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int s = *SAL_CK_LD(a.seqs + i, 4), len = *SAL_CK_LD(a.new_lengths + i, 4);
    bool wrong = s < 0 || s >= t.sequences || len < 0 || len > capacity;
    if (!wrong) wrong = (atomicOr(&listed[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u;
    if (wrong) bad = 1;
  }
  __syncthreads();
  if (bad) {
    for (int s = warp; s < t.sequences; s += kPlanThreads / 32) pass_row(t, s);
    if (tid == 0) {
      atomicOr(SAL_CK_ST(t.status, 4), SAL_CACHE_BAD_LIST);
      *SAL_CK_ST(a.count, 4) = 0;
    }
    return;
  }
  auto mark = [&](int p) {
    const uint32_t bit = 1u << (p & 31);
    if (atomicOr(&used[p >> 5], bit) & bit) atomicOr(&multi[p >> 5], bit);
  };
  for (int s = warp; s < t.sequences; s += kPlanThreads / 32) {
    if ((listed[s >> 5] >> (s & 31)) & 1u) continue;
    const int c_end = pages_of(length_of(t, s), t.page_shift);
    for (int c = lane; c < c_end; c += 32) {
      const int p = *SAL_CK_LD(t.table + static_cast<int64_t>(s) * t.max_pages + c, 4);
      if (p >= 0 && p < t.pages) mark(p);
    }
    pass_row(t, s);
  }
  for (int i = warp; i < a.n; i += kPlanThreads / 32) {
    const Entry e = entry_of(a, i);
    const int c_end = pages_of(e.kept, t.page_shift);
    for (int c = lane; c < c_end; c += 32) {
      const int p = kept_page(a, e, c);
      if (p >= 0) mark(p);
    }
  }
  __syncthreads();
  // what each entry asks for, and where its share of the free pages begins (more than there are pages
  // counts as one more, so that the sums of any list stay in 32 bits)
  int asked = 0;
  for (int base = 0; base < a.n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0, from;
    if (i < a.n) {
      const Entry e = entry_of(a, i);
      if (grows_from_lost(a, e)) lost = 1;
      need = min(pages_of(e.len, t.page_shift) - pages_of(e.kept, t.page_shift) + replaces(a, e, multi, from),
                 t.pages + 1);
    }
    int total;
    const int at = asked + block_scan(need, warp_sums, total);
    if (i < a.n) *SAL_CK_ST(a.offs + i, 4) = at;
    asked = min(asked + total, t.pages + 1);
  }
  const int chunk = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, tid * chunk), w1 = min(words, w0 + chunk);
  auto free_bits = [&](int w) {
    const int top = t.pages - 32 * w;
    return ~used[w] & (top >= 32 ? 0xffffffffu : (1u << top) - 1u);
  };
  int mine = 0, n_free;
  for (int w = w0; w < w1; ++w) mine += __popc(free_bits(w));
  int rank = block_scan(mine, warp_sums, n_free);
  if (lost || asked > n_free) {
    for (int i = warp; i < a.n; i += kPlanThreads / 32) pass_row(t, *SAL_CK_LD(a.seqs + i, 4));
    if (tid == 0) {
      atomicOr(SAL_CK_ST(t.status, 4), lost ? SAL_CACHE_LOST : SAL_CACHE_NO_PAGES);
      *SAL_CK_ST(a.count, 4) = 0;
    }
    return;
  }
  for (int w = w0; w < w1 && rank < asked; ++w)
    for (uint32_t bits = free_bits(w); bits && rank < asked; bits &= bits - 1)
      *SAL_CK_ST(a.freed + rank++, 4) = 32 * w + __ffs(bits) - 1;
  __syncthreads();
  for (int i = warp; i < a.n; i += kPlanThreads / 32) {
    const Entry e = entry_of(a, i);
    int from;
    const bool swap = replaces(a, e, multi, from);
    const int32_t* mine_free = a.freed + *SAL_CK_LD(a.offs + i, 4);
    const int c_kept = pages_of(e.kept, t.page_shift), c_new = pages_of(e.len, t.page_shift);
    const int c_swap = swap ? e.kept >> t.page_shift : -1;
    const int64_t at = static_cast<int64_t>(e.seq) * t.max_pages;
    __syncwarp();
    for (int c = lane; c < t.max_pages; c += 32) {
      int p = -1;
      if (c >= c_kept)
        p = c < c_new ? *SAL_CK_LD(mine_free + swap + (c - c_kept), 4) : -1;
      else if (c == c_swap)
        p = *SAL_CK_LD(mine_free, 4);
      else if (c < c_new)
        p = kept_page(a, e, c);
      *SAL_CK_ST(t.table_out + at + c, 4) = p;
    }
    if (lane == 0) {
      *SAL_CK_ST(t.lengths_out + e.seq, 4) = e.len;
      if (swap) *SAL_CK_ST(a.pairs + atomicAdd(&n_pairs, 1), 8) = make_int2(from, *SAL_CK_LD(mine_free, 4));
    }
  }
  __syncthreads();
  if (tid == 0) *SAL_CK_ST(a.count, 4) = n_pairs;
}

__global__ void __launch_bounds__(kPlanThreads, 1) compact_kernel(const PlanArgs a) {
  extern __shared__ uint32_t sm[];
  const TableArgs& t = a.t;
  const int words = (t.pages + 31) >> 5;
  uint32_t* used = sm;
  int* before = reinterpret_cast<int*>(sm + words);  // pages in use below each word
  __shared__ int warp_sums[33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < words; i += kPlanThreads) used[i] = 0;
  __syncthreads();
  for (int s = warp; s < t.sequences; s += kPlanThreads / 32) {
    const int c_end = pages_of(length_of(t, s), t.page_shift);
    for (int c = lane; c < c_end; c += 32) {
      const int p = *SAL_CK_LD(t.table + static_cast<int64_t>(s) * t.max_pages + c, 4);
      if (p >= 0 && p < t.pages) atomicOr(&used[p >> 5], 1u << (p & 31));
    }
  }
  __syncthreads();
  const int chunk = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, tid * chunk), w1 = min(words, w0 + chunk);
  int mine = 0, m;
  for (int w = w0; w < w1; ++w) mine += __popc(used[w]);
  int run = block_scan(mine, warp_sums, m);
  for (int w = w0; w < w1; ++w) {
    before[w] = run;
    run += __popc(used[w]);
  }
  __syncthreads();
  // pages in use below page p (p < pages)
  auto rank = [&](int p) { return before[p >> 5] + __popc(used[p >> 5] & ((1u << (p & 31)) - 1u)); };
  const int low = m < t.pages ? rank(m) : m;  // of the m pages, those that stay
  for (int p = tid; p < m; p += kPlanThreads)
    if (!((used[p >> 5] >> (p & 31)) & 1u)) *SAL_CK_ST(a.freed + (p - rank(p)), 4) = p;
  __syncthreads();
  for (int p = m + tid; p < t.pages; p += kPlanThreads)
    if ((used[p >> 5] >> (p & 31)) & 1u) {
      const int i = rank(p) - low;
      *SAL_CK_ST(a.pairs + i, 8) = make_int2(p, *SAL_CK_LD(a.freed + i, 4));
    }
  for (int s = warp; s < t.sequences; s += kPlanThreads / 32) {
    const int c_end = pages_of(length_of(t, s), t.page_shift);
    const int64_t at = static_cast<int64_t>(s) * t.max_pages;
    for (int c = lane; c < t.max_pages; c += 32) {
      int p = -1;
      if (c < c_end) {
        p = *SAL_CK_LD(t.table + at + c, 4);
        if (p < 0 || p >= t.pages)
          p = -1;
        else if (p >= m)
          p = *SAL_CK_LD(a.freed + rank(p) - low, 4);
      }
      *SAL_CK_ST(t.table_out + at + c, 4) = p;
    }
    if (lane == 0 && t.lengths_out != t.lengths) *SAL_CK_ST(t.lengths_out + s, 4) = *SAL_CK_LD(t.lengths + s, 4);
  }
  if (tid == 0) *SAL_CK_ST(a.count, 4) = m - low;
}

// fork: a block takes `cols` columns of every listed row (column max_pages is the lengths),
// reads all sources into shared memory and then writes all destinations, so a list that
// permutes the rows in place needs no second copy of the table.
__global__ void __launch_bounds__(256) fork_kernel(const TableArgs t, const int32_t* src, const int32_t* dst, int n,
                                                   int cols) {
  extern __shared__ uint32_t sm[];
  const int seq_words = (t.sequences + 31) >> 5;
  uint32_t* listed = sm;
  int32_t* tile = reinterpret_cast<int32_t*>(sm + seq_words);
  __shared__ int bad;
  const int tid = threadIdx.x, c0 = blockIdx.x * cols;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < seq_words; i += 256) listed[i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int i = tid; i < n; i += 256) {
    const int s = *SAL_CK_LD(src + i, 4), d = *SAL_CK_LD(dst + i, 4);
    bool wrong = s < 0 || s >= t.sequences || d < 0 || d >= t.sequences;
    if (!wrong) wrong = (atomicOr(&listed[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1u;
    if (wrong) bad = 1;
  }
  __syncthreads();
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(SAL_CK_ST(t.status, 4), SAL_CACHE_BAD_LIST);
  auto read = [&](int seq, int c) {
    return c < t.max_pages ? *SAL_CK_LD(t.table + static_cast<int64_t>(seq) * t.max_pages + c, 4)
                           : *SAL_CK_LD(t.lengths + seq, 4);
  };
  auto write = [&](int seq, int c, int32_t v) {
    if (c < t.max_pages)
      *SAL_CK_ST(t.table_out + static_cast<int64_t>(seq) * t.max_pages + c, 4) = v;
    else
      *SAL_CK_ST(t.lengths_out + seq, 4) = v;
  };
  const int take = min(cols, t.max_pages + 1 - c0);
  if (!bad) {
    for (int i = tid; i < n * take; i += 256) tile[i] = read(*SAL_CK_LD(src + i / take, 4), c0 + i % take);
    __syncthreads();
    for (int i = tid; i < n * take; i += 256) write(*SAL_CK_LD(dst + i / take, 4), c0 + i % take, tile[i]);
  }
  for (int c = c0; c < c0 + take; ++c) {
    if (c < t.max_pages ? t.table_out == t.table : t.lengths_out == t.lengths) continue;
    for (int s = tid; s < t.sequences; s += 256)
      if (bad || !((listed[s >> 5] >> (s & 31)) & 1u)) write(s, c, read(s, c));
  }
}

struct CopyArgs {
  uint4 *k, *v;          // pools as 16-byte vectors
  int64_t layer_vecs;    // vectors of a layer
  int page_vecs, segs;   // vectors of a page, 1024-vector segments of a page
  int pages;
  const int32_t* count;  // pairs: on the device (plan) or n
  const int2* pairs;
  const int32_t *src, *dst;
  int n;
  uint32_t* status;
};

// Whole pages, 16 KB of one page per block and step: blockIdx.y names the layer and the pool.
__global__ void __launch_bounds__(256) copy_pages_kernel(const CopyArgs a) {
  pdl_wait();
  pdl_trigger();
  const unsigned total = static_cast<unsigned>(a.count ? *SAL_CK_LD(a.count, 4) : a.n) * a.segs;
  uint4* pool = (blockIdx.y & 1 ? a.v : a.k) + (blockIdx.y >> 1) * a.layer_vecs;
  for (unsigned u = blockIdx.x; u < total; u += gridDim.x) {
    const unsigned i = u / a.segs;
    int2 pr;
    if (a.pairs)
      pr = *SAL_CK_LD(a.pairs + i, 8);
    else
      pr = make_int2(*SAL_CK_LD(a.src + i, 4), *SAL_CK_LD(a.dst + i, 4));
    if (pr.x < 0 || pr.x >= a.pages || pr.y < 0 || pr.y >= a.pages) {
      if (threadIdx.x == 0) atomicOr(SAL_CK_ST(a.status, 4), SAL_CACHE_BAD_LIST);
      continue;
    }
    const int base = static_cast<int>(u - i * a.segs) * 1024 + threadIdx.x;
    const uint4* from = pool + static_cast<int64_t>(pr.x) * a.page_vecs;
    uint4* to = pool + static_cast<int64_t>(pr.y) * a.page_vecs;
    uint4 x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (base + 256 * r < a.page_vecs) x[r] = *SAL_CK_LD(from + base + 256 * r, 16);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (base + 256 * r < a.page_vecs) *SAL_CK_ST(to + base + 256 * r, 16) = x[r];
  }
}

struct AppendArgs {
  const uint4 *k, *v;  // [batch, kv_heads, T] rows of row_vecs vectors
  uint4 *k_pages, *v_pages;
  const int32_t *table, *lengths, *starts, *seqs;
  const uint32_t* failed;  // nothing is written where this is set (may be null)
  int T, kv_heads, row_shift;  // row_vecs = 1 << row_shift
  int sequences, max_pages, pages, page_shift;
};

__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  if (a.failed && *SAL_CK_LD(a.failed, 4)) return;
  const int b = blockIdx.y;
  const int seq = a.seqs ? *SAL_CK_LD(a.seqs + b, 4) : b;
  if (seq < 0 || seq >= a.sequences) return;
  const int len = min(*SAL_CK_LD(a.lengths + seq, 4), a.max_pages << a.page_shift);
  const int start = a.starts ? *SAL_CK_LD(a.starts + b, 4) : 0;
  const unsigned per_row = static_cast<unsigned>(a.kv_heads) * a.T;  // (head, token) rows of this batch row
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  const unsigned r = i >> a.row_shift, c = i & ((1u << a.row_shift) - 1);
  if (r >= per_row) return;
  const unsigned h = r / a.T;
  const int64_t p = static_cast<int64_t>(start) + (r - h * a.T);
  if (p < 0 || p >= len) return;
  const int page = *SAL_CK_LD(a.table + static_cast<int64_t>(seq) * a.max_pages + (p >> a.page_shift), 4);
  if (page < 0 || page >= a.pages) return;
  const int64_t from = ((static_cast<int64_t>(b) * per_row + r) << a.row_shift) + c;
  const int64_t slot = (((static_cast<int64_t>(page) * a.kv_heads + h) << a.page_shift) +
                        (p & ((1 << a.page_shift) - 1)));
  const int64_t to = (slot << a.row_shift) + c;
  const uint4 x = *SAL_CK_LD(a.k + from, 16), y = *SAL_CK_LD(a.v + from, 16);
  *SAL_CK_ST(a.k_pages + to, 16) = x;
  *SAL_CK_ST(a.v_pages + to, 16) = y;
}

std::mutex g_mu;
bool g_attr[64] = {};

// Lets the plan and fork kernels use all the shared memory their largest case takes.
sal_status kernel_attributes() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SAL_ECUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_attr[dev]) {
    const int most = 4 * (2 * SAL_CACHE_MAX_PAGES / 32 + SAL_CACHE_MAX_SEQUENCES / 32);
    if (cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (kForkInts + SAL_CACHE_MAX_SEQUENCES / 32)) != cudaSuccess)
      return SAL_ECUDA;
    g_attr[dev] = true;
  }
  return SAL_OK;
}

TableArgs table_args(const sal_cache* c, int32_t* table_out, int32_t* lengths_out) {
  return TableArgs{c->table,     c->lengths,   table_out, lengths_out, c->status,
                   c->sequences, c->max_pages, c->pages,  __builtin_ctz(static_cast<unsigned>(c->page_size))};
}

PlanArgs plan_args(const sal_cache* c, int32_t* table_out, int32_t* lengths_out) {
  const Layout l = ws_layout(c->pages, c->sequences);
  char* w = static_cast<char*>(c->workspace);
  PlanArgs a{};
  a.t = table_args(c, table_out, lengths_out);
  a.left = -1;
  a.count = reinterpret_cast<int32_t*>(w);
  a.pairs = reinterpret_cast<int2*>(w + l.pairs);
  a.freed = reinterpret_cast<int32_t*>(w + l.freed);
  a.offs = reinterpret_cast<int32_t*>(w + l.offs);
  return a;
}

void declare_tables(const TableArgs& t) {
  const uint64_t tb = static_cast<uint64_t>(t.sequences) * t.max_pages * 4, lb = static_cast<uint64_t>(t.sequences) * 4;
  ck_declare(t.table, tb, t.table_out == t.table);
  ck_declare(t.lengths, lb, t.lengths_out == t.lengths);
  if (t.table_out != t.table) ck_declare(t.table_out, tb, true);
  if (t.lengths_out != t.lengths) ck_declare(t.lengths_out, lb, true);
  ck_declare(t.status, 4, true);
}

// The copy behind a plan (pairs == nullptr: behind no plan, n pairs of src and dst).
sal_status copy_launch(const sal_cache* c, const PlanArgs* plan, const int32_t* src, const int32_t* dst, int n,
                       cudaStream_t s) {
  CopyArgs a{};
  a.k = static_cast<uint4*>(c->k);
  a.v = static_cast<uint4*>(c->v);
  a.page_vecs = c->kv_heads * c->page_size * (c->head_dim / 8);
  a.layer_vecs = static_cast<int64_t>(c->pages) * a.page_vecs;
  a.segs = (a.page_vecs + 1023) / 1024;
  a.pages = c->pages;
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.status = c->status;
  if (plan) {
    a.count = plan->count;
    a.pairs = plan->pairs;
    ck_declare(a.count, 4, false);
    ck_declare(a.pairs, static_cast<uint64_t>(c->pages) * 8, false);
  } else {
    ck_declare(src, static_cast<uint64_t>(n) * 4, false);
    ck_declare(dst, static_cast<uint64_t>(n) * 4, false);
  }
  const uint64_t pool = static_cast<uint64_t>(c->layers) * a.layer_vecs * 16;
  ck_declare(a.k, pool, true);
  ck_declare(a.v, pool, true);
  ck_declare(a.status, 4, true);
  const int slots = 148 * 8;  // blocks that fit at once
  const dim3 grid(static_cast<unsigned>(std::max(1, (slots + 2 * c->layers - 1) / (2 * c->layers))),
                  static_cast<unsigned>(2 * c->layers));
  return launch_kernel(copy_pages_kernel, grid, dim3(256), 0, s, a) == cudaSuccess ? SAL_OK : SAL_ECUDA;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

sal_status check_cache(const sal_cache* c, bool workspace) {
  if (!c || c->layers < 0 || c->pages < 0 || c->kv_heads < 0 || c->sequences < 0 || c->max_pages < 0)
    return SAL_EINVAL;
  if (c->layers < 1 || c->layers > 32767 || c->pages < 1 || c->pages > SAL_CACHE_MAX_PAGES || c->kv_heads < 1 ||
      c->kv_heads > 65535 || c->sequences < 1 || c->sequences > SAL_CACHE_MAX_SEQUENCES || c->max_pages < 1 ||
      c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) ||
      (c->head_dim != 64 && c->head_dim != 128) ||
      static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 28))
    return SAL_ESHAPE;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v) || !c->table || !aligned4(c->table) || !c->lengths ||
      !aligned4(c->lengths) || !c->status || !aligned4(c->status))
    return SAL_EINVAL;
  if (workspace) {
    if (!c->workspace || (reinterpret_cast<uintptr_t>(c->workspace) & 255u)) return SAL_EINVAL;
    if (c->workspace_bytes < ws_layout(c->pages, c->sequences).bytes) return SAL_EWORKSPACE;
  }
  return SAL_OK;
}

}  // namespace sal

using namespace sal;

#define SAL_TRY(expr)              \
  do {                             \
    const sal_status st_ = (expr); \
    if (st_ != SAL_OK) return st_; \
  } while (0)

sal_status sal::cache_append(const sal_cache* cache, int layer, const void* k, const void* v, int batch, int64_t T,
                             const int32_t* starts, const int32_t* seqs, bool unless_failed, cudaStream_t s) {
  SAL_TRY(check_cache(cache, false));
  if (batch < 0 || T < 0 || layer < 0 || layer >= cache->layers) return SAL_EINVAL;
  const int row_shift = cache->head_dim == 128 ? 4 : 3;
  if (batch > 65535 || T > (int64_t(1) << 28) || ((cache->kv_heads * T) << row_shift) > (int64_t(1) << 31))
    return SAL_ESHAPE;
  if (batch == 0 || T == 0) return SAL_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !aligned4(starts) || !aligned4(seqs)) return SAL_EINVAL;
  if (!seqs && batch > cache->sequences) return SAL_EINVAL;
  SAL_TRY(require_device());
  AppendArgs a{};
  const int64_t layer_vecs = (static_cast<int64_t>(cache->pages) * cache->kv_heads * cache->page_size) << row_shift;
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.k_pages = static_cast<uint4*>(cache->k) + layer * layer_vecs;
  a.v_pages = static_cast<uint4*>(cache->v) + layer * layer_vecs;
  a.table = cache->table;
  a.lengths = cache->lengths;
  a.starts = starts;
  a.seqs = seqs;
  a.failed = unless_failed ? cache->status : nullptr;
  a.T = static_cast<int>(T);
  a.kv_heads = cache->kv_heads;
  a.row_shift = row_shift;
  a.sequences = cache->sequences;
  a.max_pages = cache->max_pages;
  a.pages = cache->pages;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(cache->page_size));
  const int64_t row_vecs = (cache->kv_heads * T) << row_shift;
  ck_declare(k, batch * row_vecs * 16, false);
  ck_declare(v, batch * row_vecs * 16, false);
  ck_declare(a.k_pages, layer_vecs * 16, true);
  ck_declare(a.v_pages, layer_vecs * 16, true);
  ck_declare(a.table, static_cast<uint64_t>(a.sequences) * a.max_pages * 4, false);
  ck_declare(a.lengths, static_cast<uint64_t>(a.sequences) * 4, false);
  ck_declare(starts, static_cast<uint64_t>(batch) * 4, false);
  ck_declare(seqs, static_cast<uint64_t>(batch) * 4, false);
  ck_declare(a.failed, 4, false);
  const dim3 grid(static_cast<unsigned>((row_vecs + 255) / 256), static_cast<unsigned>(batch));
  return launch_kernel(append_kernel, grid, dim3(256), 0, s, a) == cudaSuccess
             ? SAL_OK
             : SAL_ECUDA;
}

extern "C" {

size_t sal_cache_workspace_bytes(int pages, int sequences) {
  if (pages <= 0 || sequences <= 0) return 0;
  return ws_layout(pages, sequences).bytes;
}

sal_status sal_cache_append(const sal_cache* cache, int layer, const void* k, const void* v, int batch, int64_t T,
                            const int32_t* starts, const int32_t* seqs, void* stream) {
  const NvtxRange nvtx_("sal_cache_append");
  return cache_append(cache, layer, k, v, batch, T, starts, seqs, false, static_cast<cudaStream_t>(stream));
}

sal_status sal_cache_copy_pages(const sal_cache* cache, const int32_t* src, const int32_t* dst, int n, void* stream) {
  const NvtxRange nvtx_("sal_cache_copy_pages");
  SAL_TRY(check_cache(cache, false));
  if (n < 0 || n > cache->pages) return SAL_EINVAL;
  if (n == 0) return SAL_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst)) return SAL_EINVAL;
  SAL_TRY(require_device());
  return copy_launch(cache, nullptr, src, dst, n, static_cast<cudaStream_t>(stream));
}

sal_status sal_cache_fork(const sal_cache* cache, const int32_t* src, const int32_t* dst, int n, int32_t* table_out,
                          int32_t* lengths_out, void* stream) {
  const NvtxRange nvtx_("sal_cache_fork");
  SAL_TRY(check_cache(cache, false));
  if (n < 0 || n > cache->sequences) return SAL_EINVAL;
  if (!table_out || !lengths_out || !aligned4(table_out) || !aligned4(lengths_out)) return SAL_EINVAL;
  if (n > 0 && (!src || !dst || !aligned4(src) || !aligned4(dst))) return SAL_EINVAL;
  SAL_TRY(require_device());
  SAL_TRY(kernel_attributes());
  const TableArgs t = table_args(cache, table_out, lengths_out);
  // as many blocks as keep a thread at one or two entries of the list's columns
  const int cols = std::max(1, std::min(32, n > 0 ? 512 / n : 32));
  declare_tables(t);
  ck_declare(src, static_cast<uint64_t>(n) * 4, false);
  ck_declare(dst, static_cast<uint64_t>(n) * 4, false);
  const size_t smem = 4 * (static_cast<size_t>((t.sequences + 31) / 32) + static_cast<size_t>(n) * cols);
  return launch_kernel(fork_kernel, dim3(static_cast<unsigned>((t.max_pages + cols) / cols)), dim3(256), smem,
                       static_cast<cudaStream_t>(stream), t, src, dst, n, cols) == cudaSuccess
             ? SAL_OK
             : SAL_ECUDA;
}

sal_status sal_cache_resize(const sal_cache* cache, const int32_t* seqs, const int32_t* new_lengths, int n,
                            const sal_window* window, int32_t* table_out, int32_t* lengths_out, void* stream) {
  const NvtxRange nvtx_("sal_cache_resize");
  SAL_TRY(check_cache(cache, true));
  if (n < 0 || n > cache->sequences || (window && window->sinks < 0)) return SAL_EINVAL;
  if (!table_out || !lengths_out || !aligned4(table_out) || !aligned4(lengths_out)) return SAL_EINVAL;
  if (n > 0 && (!seqs || !new_lengths || !aligned4(seqs) || !aligned4(new_lengths))) return SAL_EINVAL;
  SAL_TRY(require_device());
  SAL_TRY(kernel_attributes());
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PlanArgs a = plan_args(cache, table_out, lengths_out);
  a.seqs = seqs;
  a.new_lengths = new_lengths;
  a.n = n;
  if (window && window->left >= 0) {
    const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
    a.left = static_cast<int>(std::min(window->left, cap));
    a.sinks = static_cast<int>(std::min(window->sinks, cap));
  }
  declare_tables(a.t);
  ck_declare(seqs, static_cast<uint64_t>(n) * 4, false);
  ck_declare(new_lengths, static_cast<uint64_t>(n) * 4, false);
  ck_declare(cache->workspace, cache->workspace_bytes, true);
  const int words = (cache->pages + 31) / 32;
  const size_t smem = 4 * (2 * static_cast<size_t>(words) + (cache->sequences + 31) / 32);
  if (launch_kernel(resize_kernel, dim3(1), dim3(kPlanThreads), smem, s, a) != cudaSuccess) return SAL_ECUDA;
  return copy_launch(cache, &a, nullptr, nullptr, 0, s);
}

sal_status sal_cache_compact(const sal_cache* cache, int32_t* table_out, int32_t* lengths_out, void* stream) {
  const NvtxRange nvtx_("sal_cache_compact");
  SAL_TRY(check_cache(cache, true));
  if (!table_out || !lengths_out || !aligned4(table_out) || !aligned4(lengths_out)) return SAL_EINVAL;
  SAL_TRY(require_device());
  SAL_TRY(kernel_attributes());
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PlanArgs a = plan_args(cache, table_out, lengths_out);
  declare_tables(a.t);
  ck_declare(cache->workspace, cache->workspace_bytes, true);
  const size_t smem = 8 * static_cast<size_t>((cache->pages + 31) / 32);
  if (launch_kernel(compact_kernel, dim3(1), dim3(kPlanThreads), smem, s, a) != cudaSuccess) return SAL_ECUDA;
  return copy_launch(cache, &a, nullptr, nullptr, 0, s);
}

}  // extern "C"
