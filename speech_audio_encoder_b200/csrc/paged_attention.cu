// Attention of one new position per sequence over a paged key/value cache (sal_attention_paged):
// row b's query is position p = n - 1 of its sequence of n positions, and
//   o[b, h, :] = sum_j a_j v_j,  a = softmax_j(q k_j / sqrt(d)) over the keys j < n with
//   j >= p - left or j < sinks, whose page the table still names.
//
// Bound by memory: every visible key and value is read once, 4 d bytes for 4 d flops of each
// query head that shares it. A warp takes 16 keys at a time through its own ring of asynchronous
// 16-byte copies (no barrier between warps), multiplies up to 16 query rows - the heads that
// share the key head - with them by warp-level matrix products, and keeps a running maximum and
// sum in fp32; the products cost a tenth of the copies' time whether 1 or 16 of the rows are
// real, so one form serves every grouping. Keys that the mask hides are not read (their place
// is filled with zeros, so nothing that memory holds there can reach a sum).
// The weights are rounded to bf16 for the product with V (the sum of weights is not); sums,
// maxima and the joined pieces are fp32.
//
// The key axis is split, by one of two rules (plan_of):
//   * few keys: a cluster per row and key head, joined through shared memory, one launch;
//   * many: all rows' keys in one line cut into equal parts; the pieces of a row are joined by the
//     block that brings the last of them, or by a second small kernel.
// Measured on one B200 with inputs larger than L2: 64 rows of up to 8,190 keys (10 heads of 128)
// 265-270 us, 6.2-6.3 TB/s, 95-97 % of a plain copy's rate; 64 rows that see 758 of their 45,000 keys
// 50 us, of which 38 are bytes and the rest the start of a block's copies (page table, then keys) and
// its end; 3 rows of up to 45,000 keys, 32 heads on 2, 30 us: 14 bytes, 3 to start, 3 to
// merge the warps, 5 for the join. One row of 750 keys is 6 us on the device as clusters and 11 as
// a line. Three blocks on an SM with two stages each changed none of it.
#define SAL_CK_FILE 7
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <functional>
#include <mutex>

#include "sal_internal.h"
#include "sal_mma.cuh"

namespace sal {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;                // keys of a block: one matrix-product depth
constexpr int kRowTile = 16;             // query rows of a block: the heads that share a key head
constexpr int kClusterSplits = 8;        // splits that join inside a cluster
constexpr int kSlots = 148 * 2;          // blocks that fit on the GPU at once
constexpr int kFewKeys = 8;              // blocks of keys below which a split is not worth its start
// The least maximum of a row that has seen a key: scores of -infinity are then weights of zero (minus
// a maximum of -infinity they would be NaN), and a maximum of -infinity means that nothing is visible.
constexpr float kLeastMax = -3.402823466e38f;

template <int HD>
struct Ring {
  static constexpr int kRow = HD * 2;                    // bytes of a key
  static constexpr int kHalf = kKeys * kRow;             // K (or V) of a block of keys
  static constexpr int kStages = HD == 128 ? 3 : 6;
  static constexpr int kBytes = kWarps * kStages * 2 * kHalf;
  static constexpr int kPitch = HD + 4;                  // floats between merged rows
  static_assert((kWarps * kRowTile * (kPitch + 2) + 2 * kRowTile) * 4 <= kBytes, "the merge fits in the ring");
};

struct PagedArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  float* part;    // [grid][2][16 rows][head_dim]: the sums of a block's pieces
  float2* stats;  // [grid][2][16 rows]: their maximum and total weight
  // what was cut into pieces: (row, group, first part, pieces; 0: nothing to join), by its place
  // among all (row, group) pairs, or by its first part where there are fewer of those
  int4* joins;
  int by_part;
  int* arrived;  // [grid] pieces that are there of what begins in a part: zero between calls
  int inside;    // the last piece's block joins them; else paged_join_kernel does
  int64_t q_row, q_head;
  const int32_t *table, *lengths, *seqs;
  int batch, heads, kv_heads, row_tiles, pages, page_shift, sequences, max_pages;
  int left, sinks, splits;
  float scale_log2;
};

// The visible keys of a row: positions [low, n) and [0, sinks), in blocks of 16 from position 0.
// Blocks [0, first) hold the sinks, blocks [second, second + rest) the window.
struct Span {
  int n, low, sinks, first, second, blocks;
  __device__ int block(int i) const { return i < first ? i : second + (i - first); }
};
__device__ __forceinline__ Span span_of(const PagedArgs& a, int seq) {
  Span s;
  s.n = 0;
  if (seq >= 0 && seq < a.sequences) s.n = min(max(*SAL_CK_LD(a.lengths + seq, 4), 0), a.max_pages << a.page_shift);
  s.low = max(0, s.n - 1 - a.left);
  s.sinks = min(a.sinks, s.low);
  s.first = (s.sinks + kKeys - 1) / kKeys;
  s.second = max(s.low / kKeys, s.first);
  s.blocks = s.first + (s.n + kKeys - 1) / kKeys - s.second;
  return s;
}

// One row's (or heads') share of the keys, blocks [lo, hi) of its span: every warp takes each
// fourth block through its own ring of copies and leaves its rows' sums in shared memory,
// [warps][16][pitch] and behind them (maximum, total) [warps][16][2]. All threads call it; on
// return the results are visible to all of them.
template <int HD>
__device__ __forceinline__ void walk(const PagedArgs& a, const Span& sp, int seq, int b, int kvh, int h0, int rows,
                                     int lo, int hi, uint8_t* smem) {
  using R = Ring<HD>;
  constexpr int C = HD / 8;            // 16-byte chunks of a key
  constexpr int kIts = kKeys * C / 32;  // copies per lane of K (or V)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = max(0, (hi - lo - warp + kWarps - 1) / kWarps);  // blocks lo + warp + 4 t of this warp
  const int32_t* row = a.table + static_cast<int64_t>(seq) * a.max_pages;
  const int mask = (1 << a.page_shift) - 1;

  // Table entries of the warp's blocks 32 g + lane, both halves (a page of 8 ends mid-block).
  auto entries = [&](int g, int& e0, int& e1) {
    e0 = e1 = -1;
    const int t = 32 * g + lane;
    if (t >= nt) return;
    const int base = sp.block(lo + warp + kWarps * t) * kKeys;
    e0 = *SAL_CK_LD(row + (base >> a.page_shift), 4);
    e1 = e0;
    if (a.page_shift == 3) e1 = base + 8 < sp.n ? *SAL_CK_LD(row + (base >> 3) + 1, 4) : -1;
    if (static_cast<unsigned>(e0) >= static_cast<unsigned>(a.pages)) e0 = -1;
    if (static_cast<unsigned>(e1) >= static_cast<unsigned>(a.pages)) e1 = -1;
  };
  int cur0, cur1, next0, next1;
  entries(0, cur0, cur1);
  entries(1, next0, next1);
  const uint32_t ring = smem_u32(smem) + warp * (R::kStages * 2 * R::kHalf);
  const int chunk = lane % C, row_in = lane / C;
  uint32_t bad0 = 0, bad1 = 0;  // bit t % 32: the halves of block t that have no page (of the issued ones)

  auto issue = [&](int t) {
    if (t < nt) {
      if ((t & 31) == 0 && t > 0) {
        cur0 = next0;
        cur1 = next1;
        entries(t / 32 + 1, next0, next1);
      }
      const int e0 = __shfl_sync(0xffffffffu, cur0, t & 31), e1 = __shfl_sync(0xffffffffu, cur1, t & 31);
      bad0 = (bad0 & ~(1u << (t & 31))) | (static_cast<uint32_t>(e0 < 0) << (t & 31));
      bad1 = (bad1 & ~(1u << (t & 31))) | (static_cast<uint32_t>(e1 < 0) << (t & 31));
      const int base = sp.block(lo + warp + kWarps * t) * kKeys;
      const uint32_t dst = ring + (t % R::kStages) * (2 * R::kHalf);
      const int64_t at0 = ((static_cast<int64_t>(max(e0, 0)) * a.kv_heads + kvh) << a.page_shift) + (base & mask);
      const int64_t at1 = ((static_cast<int64_t>(max(e1, 0)) * a.kv_heads + kvh) << a.page_shift) + ((base + 8) & mask);
#pragma unroll
      for (int i = 0; i < kIts; ++i) {
        const int r = row_in + (32 / C) * i;  // rows 0..7 in the first half of the copies
        const int pos = base + r;
        const bool fill = pos < sp.n && (pos >= sp.low || pos < sp.sinks) && (i < kIts / 2 ? e0 : e1) >= 0;
        const int64_t at = ((i < kIts / 2 ? at0 : at1 - 8) + r) * HD + chunk * 8;
        const uint32_t to = dst + r * R::kRow + ((chunk ^ (r & 7)) << 4);
        cp_async16(to, fill ? SAL_CK_LD(a.k + at, 16) : a.k, fill);
        cp_async16(to + R::kHalf, fill ? SAL_CK_LD(a.v + at, 16) : a.v, fill);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int t = 0; t < R::kStages - 1; ++t) issue(t);

  // the query rows as matrix fragments: lane l holds columns 2 (l % 4) + {0, 1, 8, 9} of rows l / 4 and l / 4 + 8
  const int g = lane >> 2, quad = lane & 3;
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = g + 8 * (e & 1), d = kk * 16 + quad * 2 + 8 * (e >> 1);
      qf[kk][e] = 0;
      if (r < rows)
        qf[kk][e] = *SAL_CK_LD(reinterpret_cast<const uint32_t*>(a.q + b * a.q_row + (h0 + r) * a.q_head + d), 4);
    }
  float acc[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int t = 0; t < nt; ++t) {
    issue(t + R::kStages - 1);
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const int base = sp.block(lo + warp + kWarps * t) * kKeys;
    // visible keys of the block: below n, not between the sinks and the window, with a page
    uint32_t vis = 0xffffu;
    if (sp.n - base < kKeys) vis &= (1u << (sp.n - base)) - 1u;
    const int h_lo = min(max(sp.sinks - base, 0), kKeys), h_hi = min(max(sp.low - base, 0), kKeys);
    if (h_hi > h_lo) vis &= ~(((1u << h_hi) - 1u) & ~((1u << h_lo) - 1u));
    if ((bad0 >> (t & 31)) & 1u) vis &= 0xff00u;
    if ((bad1 >> (t & 31)) & 1u) vis &= 0x00ffu;
    if (vis) {
      const uint32_t sk = ring + (t % R::kStages) * (2 * R::kHalf), sv = sk + R::kHalf;
      float s[2][4] = {};
      const int k_key = (lane >> 4) * 8 + (lane & 7), k_chunk = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        uint32_t kf[4];
        ldmatrix4(kf, sk + k_key * R::kRow + (((2 * kk + k_chunk) ^ (k_key & 7)) << 4));
        mma_bf16(s[0], qf[kk], kf[0], kf[1]);
        mma_bf16(s[1], qf[kk], kf[2], kf[3]);
      }
      if (vis != 0xffffu) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((vis >> (8 * i + 2 * quad + (e & 1))) & 1u)) s[i][e] = -INFINITY;
      }
      float p[2][4], fac[2];
      bool grew = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx * a.scale_log2, kLeastMax);
        fac[r] = 1.f;
        if (mx > m[r]) {
          fac[r] = fast_exp2(m[r] - mx);
          m[r] = mx;
          grew = true;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[i][2 * r + e] = fast_exp2(fmaf(s[i][2 * r + e], a.scale_log2, -m[r]));
        l[r] = l[r] * fac[r] + (p[0][2 * r] + p[0][2 * r + 1]) + (p[1][2 * r] + p[1][2 * r + 1]);
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          acc[i][0] *= fac[0];
          acc[i][1] *= fac[0];
          acc[i][2] *= fac[1];
          acc[i][3] *= fac[1];
        }
      }
      const uint32_t pf[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                              pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3])};
      const int v_key = lane & 15, v_chunk = lane >> 4;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        uint32_t vf[4];
        ldmatrix4_trans(vf, sv + v_key * R::kRow + (((2 * i + v_chunk) ^ (v_key & 7)) << 4));
        mma_bf16(acc[2 * i], pf, vf[0], vf[1]);
        mma_bf16(acc[2 * i + 1], pf, vf[2], vf[3]);
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its part of the ring

  // the warps' results side by side in shared memory, then merged
  float* so = reinterpret_cast<float*>(smem);               // [warps][16][pitch]
  float* sml = so + kWarps * kRowTile * R::kPitch;          // [warps][16][2]
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int at = warp * kRowTile + g + 8 * r;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
      *reinterpret_cast<float2*>(so + at * R::kPitch + 8 * i + 2 * quad) = make_float2(acc[i][2 * r], acc[i][2 * r + 1]);
    if (quad == 0) {
      sml[2 * at] = m[r];
      sml[2 * at + 1] = l[r];
    }
  }
  __syncthreads();
}

// The warps' results of a walk into one: a weight for every warp and row, and the row's maximum and
// total weight, worked out once (by a thread per row) for all columns. All threads call it.
struct Merged {
  float weight[kRowTile][kWarps], top[kRowTile], total[kRowTile];
};
template <int HD>
__device__ __forceinline__ void merge_weights(const uint8_t* smem, int rows, Merged& m) {
  const float* sml = reinterpret_cast<const float*>(smem) + kWarps * kRowTile * Ring<HD>::kPitch;
  const int r = threadIdx.x;
  if (r < rows) {
    float mm = -INFINITY, total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[2 * (w * kRowTile + r)]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int at = w * kRowTile + r;
      const float f = sml[2 * at] != -INFINITY ? fast_exp2(sml[2 * at] - mm) : 0.f;
      total += sml[2 * at + 1] * f;
      m.weight[r][w] = f;
    }
    m.top[r] = mm;
    m.total[r] = total;
  }
  __syncthreads();
}
// Column d of row r, relative to its maximum.
template <int HD>
__device__ __forceinline__ float merged(const uint8_t* smem, const Merged& m, int r, int d) {
  const float* so = reinterpret_cast<const float*>(smem) + r * Ring<HD>::kPitch + d;
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) x = fmaf(so[w * kRowTile * Ring<HD>::kPitch], m.weight[r][w], x);
  return x;
}

// a / b for a >= 0, b > 0: in 32 bits where they fit (a tenth of the 64-bit division's time).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A row that sees nothing (its maximum is -infinity) is zeros. A total that is no number, from a query,
// key or value that is none, is stored as such, and so is 0 / 0 where every visible score is -infinity.
template <int HD>
__device__ __forceinline__ void store_out(const PagedArgs& a, int b, int h, int d, float x, float total, float top) {
  *SAL_CK_ST(a.o + (static_cast<int64_t>(b) * a.heads + h) * HD + d, 2) =
      __float2bfloat16(top == -INFINITY ? 0.f : x / total);
}

// Few keys: one cluster per (row, heads of a key head), its blocks each a split of the keys,
// joined through the cluster's shared memory. One launch and no memory traffic but the keys'.
template <int HD>
__global__ void __launch_bounds__(kThreads, 2) paged_cluster_kernel(const PagedArgs a) {
  using R = Ring<HD>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int split = blockIdx.x, group = blockIdx.y, b = blockIdx.z;
  const int kvh = group / a.row_tiles, share = a.heads / a.kv_heads;
  const int r0 = (group - kvh * a.row_tiles) * kRowTile;  // first of this block's rows among the share
  const int rows = min(kRowTile, share - r0), h0 = kvh * share + r0;
  pdl_wait();
  pdl_trigger();
  const int seq = a.seqs ? *SAL_CK_LD(a.seqs + b, 4) : b;
  const Span sp = span_of(a, seq);
  walk<HD>(a, sp, seq, b, kvh, h0, rows, sp.blocks * split / a.splits, sp.blocks * (split + 1) / a.splits, smem);
  __shared__ Merged mg;
  merge_weights<HD>(smem, rows, mg);
  // each thread: one column of every (128 / HD)-th row
  float* so = reinterpret_cast<float*>(smem);
  float* sml = so + kWarps * kRowTile * R::kPitch + 2 * kWarps * kRowTile;  // behind the warps' pairs
  const int d = threadIdx.x % HD;
  for (int r = threadIdx.x / HD; r < rows; r += kThreads / HD) {
    const float x = merged<HD>(smem, mg, r, d), mm = mg.top[r], total = mg.total[r];
    if (a.splits == 1) {
      store_out<HD>(a, b, h0 + r, d, x, total, mm);
      continue;
    }
    so[r * R::kPitch + d] = x;  // this thread alone has read column d of row r
    if (d == 0) {
      sml[2 * r] = mm;
      sml[2 * r + 1] = total;
    }
  }
  if (a.splits == 1) return;
  cluster_barrier();
  for (int r = split * (kThreads / HD) + threadIdx.x / HD; r < rows; r += a.splits * (kThreads / HD)) {
    const uint32_t at = smem_u32(sml + 2 * r), xo = smem_u32(so + r * R::kPitch + d);
    float mm = -INFINITY, x = 0.f, total = 0.f;
    for (int w = 0; w < a.splits; ++w) mm = fmaxf(mm, ld_cluster_f32(at, w));
    for (int w = 0; w < a.splits; ++w) {
      const float mw = ld_cluster_f32(at, w), f = mw != -INFINITY ? fast_exp2(mw - mm) : 0.f;
      total += ld_cluster_f32(at + 4, w) * f;
      x += ld_cluster_f32(xo, w) * f;
    }
    store_out<HD>(a, b, h0 + r, d, x, total, mm);
  }
  cluster_barrier();  // nobody's shared memory goes away while another block reads it
}

// Many keys: the blocks of keys of all rows and key heads in one line, cut into equal parts,
// one for each block that fits on the GPU, so that rows of any lengths keep every SM busy to
// the end. A part may end one row's keys and begin another's: what lies wholly inside a part is
// written out, the at most two pieces that do not go to the workspace, and the block that brings
// the last piece of a row, or paged_join_kernel, puts them together in their order, so the
// result does not depend on which came last. The lengths are on the device, so every block adds them up for itself.
template <int HD>
__global__ void __launch_bounds__(kThreads, 2) paged_line_kernel(const PagedArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[kWarps];
  __shared__ int64_t found[2];  // where the part's first row begins, and which row it is
  __shared__ int last_here;
  __shared__ Merged mg;
  const int tid = threadIdx.x, groups = a.kv_heads * a.row_tiles, share = a.heads / a.kv_heads;
  pdl_wait();
  pdl_trigger();
  auto seq_of = [&](int b) { return a.seqs ? *SAL_CK_LD(a.seqs + b, 4) : b; };
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of(a, seq_of(b)).blocks;
  int64_t upto = mine;  // with the threads before this one
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, i);
    if ((tid & 31) >= i) upto += y;
  }
  if ((tid & 31) == 31) sums[tid >> 5] = upto;
  __syncthreads();
  int64_t before = upto - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < tid >> 5) before += sums[w];
    all += sums[w];
  }
  const int64_t units = all * groups;
  // parts of at least kFewKeys blocks
  const int parts = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (units + kFewKeys - 1) / kFewKeys));
  const int c = blockIdx.x;
  const int64_t u0 = c < parts ? quotient(units * c, parts) : 0, u1 = c < parts ? quotient(units * (c + 1), parts) : 0;
  if (u0 < u1 && u0 >= before * groups && u0 < (before + mine) * groups) {
    int64_t at = before * groups;
    if (per == 1) {  // this thread's only row
      found[0] = at;
      found[1] = b0;
    }
    for (int b = b0; per > 1 && b < b1; ++b) {
      const int64_t n = static_cast<int64_t>(span_of(a, seq_of(b)).blocks) * groups;
      if (u0 < at + n) {
        found[0] = at;
        found[1] = b;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int4 join = make_int4(0, 0, 0, 0);  // by_part: what begins in this part and ends in a later one
  if (u0 < u1) {
    int64_t at = found[0], u = u0;
    int b = static_cast<int>(found[1]);
    while (u < u1) {
      const int seq = seq_of(b);
      const Span sp = span_of(a, seq);
      if (u >= at + static_cast<int64_t>(sp.blocks) * groups) {  // the next row (this one is done or has no keys)
        at += static_cast<int64_t>(sp.blocks) * groups;
        ++b;
        continue;
      }
      const int group = static_cast<int>(quotient(u - at, sp.blocks));
      const int64_t begin = at + static_cast<int64_t>(group) * sp.blocks;
      const int lo = static_cast<int>(u - begin), hi = static_cast<int>(min(static_cast<int64_t>(sp.blocks), u1 - begin));
      const int kvh = group / a.row_tiles, r0 = (group - kvh * a.row_tiles) * kRowTile;
      const int rows = min(kRowTile, share - r0), h0 = kvh * share + r0;
      walk<HD>(a, sp, seq, b, kvh, h0, rows, lo, hi, smem);
      merge_weights<HD>(smem, rows, mg);
      const bool whole = lo == 0 && hi == sp.blocks;
      // the part that holds unit v: units * e / parts <= v < units * (e + 1) / parts
      auto part_of = [&](int64_t v) {
        int64_t e = quotient(v * parts, units);
        while (quotient(units * (e + 1), parts) <= v) ++e;
        while (quotient(units * e, parts) > v) --e;
        return static_cast<int>(e);
      };
      const int from = whole || lo == 0 ? c : part_of(begin);
      const int pieces = whole ? 0 : part_of(begin + sp.blocks - 1) - from + 1;
      if (lo == 0 && !a.inside) {
        const int4 cut = make_int4(b, group, c, pieces);
        if (!whole) join = cut;
        if (tid == 0 && !a.by_part) *SAL_CK_ST(a.joins + b * groups + group, 16) = cut;
      }
      const int d = tid % HD;
      for (int r = tid / HD; r < rows; r += kThreads / HD) {
        const float x = merged<HD>(smem, mg, r, d), mm = mg.top[r], total = mg.total[r];
        if (whole) {
          store_out<HD>(a, b, h0 + r, d, x, total, mm);
          continue;
        }
        const int to = (2 * c + (lo == 0)) * kRowTile + r;
        *SAL_CK_ST(a.part + to * HD + d, 4) = x;
        if (d == 0) *SAL_CK_ST(a.stats + to, 8) = make_float2(mm, total);
      }
      if (!whole && a.inside) {
        // whichever block brings the last piece joins them all, in their order
        __threadfence();
        __syncthreads();
        if (tid == 0) last_here = atomicAdd(SAL_CK_ST(a.arrived + from, 4), 1) == pieces - 1;
        __syncthreads();
        if (last_here) {
          __threadfence();
          for (int r = tid / HD; r < rows; r += kThreads / HD) {
            float mm = -INFINITY, x = 0.f, total = 0.f;
            auto place = [&](int w) { return (2 * (from + w) + (w == 0)) * kRowTile + r; };
            for (int w = 0; w < pieces; ++w) mm = fmaxf(mm, __ldcg(SAL_CK_LD(a.stats + place(w), 8)).x);
#pragma unroll 4
            for (int w = 0; w < pieces; ++w) {
              const float2 st = __ldcg(SAL_CK_LD(a.stats + place(w), 8));
              const float f = st.x != -INFINITY ? fast_exp2(st.x - mm) : 0.f;
              total += st.y * f;
              x += __ldcg(SAL_CK_LD(a.part + place(w) * HD + d, 4)) * f;
            }
            store_out<HD>(a, b, h0 + r, d, x, total, mm);
          }
          if (tid == 0) *SAL_CK_ST(a.arrived + from, 4) = 0;
        }
      }
      u = begin + hi;
      __syncthreads();  // the merge has read what the next walk's copies overwrite
    }
  }
  if (tid == 0 && a.by_part && !a.inside) *SAL_CK_ST(a.joins + c, 16) = join;
  // rows without keys have no part: zeros
  for (int b = c; b < a.batch; b += gridDim.x)
    if (span_of(a, seq_of(b)).blocks == 0) {
      for (int i = tid; i < a.heads * HD; i += kThreads) store_out<HD>(a, b, 0, i, 0.f, 0.f, -INFINITY);
      if (!a.by_part && !a.inside)
        for (int i = tid; i < groups; i += kThreads) *SAL_CK_ST(a.joins + b * groups + i, 16) = make_int4(0, 0, 0, 0);
    }
}

// Joins the pieces of one entry of `joins`: the first part's second piece and the first
// pieces of the parts after it. One row per block: the pieces' weights first, then the lanes
// of each warp take four (or two) columns of every eighth piece.
constexpr int kJoinThreads = 256;
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedArgs a) {
  constexpr int kWide = HD / 32, kMine = (kSlots + kJoinThreads - 1) / kJoinThreads;
  __shared__ float weight[kSlots], reduced[kJoinThreads / 32], sums[kJoinThreads / 32][HD];
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int4 join = *SAL_CK_LD(a.joins + blockIdx.x, 16);
  const int share = a.heads / a.kv_heads, kvh = join.y / a.row_tiles, r0 = (join.y - kvh * a.row_tiles) * kRowTile;
  const int c = join.z, n = join.w;
  if (n == 0 || r >= min(kRowTile, share - r0)) return;
  auto piece = [&](int w) { return (2 * (c + w) + (w == 0)) * kRowTile + r; };
  float2 st[kMine];
  float mm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int w = tid + i * kJoinThreads;
    st[i] = w < n ? *SAL_CK_LD(a.stats + piece(w), 8) : make_float2(-INFINITY, 0.f);
    mm = fmaxf(mm, st[i].x);
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, i));
  if (lane == 0) reduced[warp] = mm;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) mm = fmaxf(mm, reduced[i]);
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int w = tid + i * kJoinThreads;
    if (w < n) {
      weight[w] = st[i].x != -INFINITY ? fast_exp2(st[i].x - mm) : 0.f;
      mine += st[i].y * weight[w];
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, i);
  __syncthreads();  // the weights are there, and the maxima in `reduced` have been read by all
  if (lane == 0) reduced[warp] = mine;
  float x[kWide] = {};
#pragma unroll 4
  for (int w = warp; w < n; w += kJoinThreads / 32) {
    const float f = weight[w];
    const float* from = a.part + piece(w) * HD + lane * kWide;
    if constexpr (kWide == 4) {
      const float4 v = *SAL_CK_LD(reinterpret_cast<const float4*>(from), 16);
      x[0] = fmaf(v.x, f, x[0]);
      x[1] = fmaf(v.y, f, x[1]);
      x[2] = fmaf(v.z, f, x[2]);
      x[3] = fmaf(v.w, f, x[3]);
    } else {
      const float2 v = *SAL_CK_LD(reinterpret_cast<const float2*>(from), 8);
      x[0] = fmaf(v.x, f, x[0]);
      x[1] = fmaf(v.y, f, x[1]);
    }
  }
#pragma unroll
  for (int e = 0; e < kWide; ++e) sums[warp][lane * kWide + e] = x[e];
  __syncthreads();
  if (tid >= HD) return;
  float y = 0.f, total = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    y += sums[i][tid];
    total += reduced[i];
  }
  store_out<HD>(a, join.x, kvh * share + r0 + r, tid, y, total, mm);
}

// How a call runs: clusters of `splits` blocks, or (splits == 0) a line of `grid` parts.
struct Plan {
  int row_tiles, splits, grid;
};
Plan plan_of(const sal_cache* c, int batch, int heads, int64_t keys) {
  Plan p{};
  p.row_tiles = (heads / c->kv_heads + kRowTile - 1) / kRowTile;
  const int64_t groups = static_cast<int64_t>(batch) * c->kv_heads * p.row_tiles;
  const int64_t blocks = (keys + kKeys - 1) / kKeys + 1;
  // up to 8 blocks of keys for each block of threads that fits at once, and no long axis
  if (groups * blocks <= kFewKeys * kSlots && blocks <= kClusterSplits * 4 * kFewKeys) {
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kClusterSplits, blocks / kFewKeys)));
    return p;
  }
  p.grid = static_cast<int>(std::min<int64_t>(kSlots, (groups * blocks + kFewKeys - 1) / kFewKeys));
  return p;
}

constexpr size_t kJoinBytes = (kSlots * sizeof(int4) + 255) & ~size_t(255);
constexpr size_t kArrivedBytes = (kSlots * sizeof(int) + 255) & ~size_t(255);
constexpr size_t kStatBytes = kSlots * 2 * kRowTile * sizeof(float2);
size_t workspace_bytes(int head_dim) {
  return kArrivedBytes + kJoinBytes + kStatBytes + static_cast<size_t>(kSlots) * 2 * kRowTile * head_dim * 4;
}

std::mutex g_mu;
bool g_attr[64] = {};

sal_status kernel_attributes() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SAL_ECUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_attr[dev]) {
    const auto set = [](auto kernel, int bytes) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    };
    if (!set(paged_cluster_kernel<128>, Ring<128>::kBytes) || !set(paged_line_kernel<128>, Ring<128>::kBytes) ||
        !set(paged_cluster_kernel<64>, Ring<64>::kBytes) || !set(paged_line_kernel<64>, Ring<64>::kBytes))
      return SAL_ECUDA;
    g_attr[dev] = true;
  }
  return SAL_OK;
}

template <int HD>
sal_status launch(const PagedArgs& a, const Plan& p, cudaStream_t s, const std::function<void()>& declare) {
  const unsigned groups = static_cast<unsigned>(a.kv_heads * a.row_tiles);
  declare();
  if (p.splits > 0)
    return launch_kernel_cluster(paged_cluster_kernel<HD>,
                                 dim3(static_cast<unsigned>(p.splits), groups, static_cast<unsigned>(a.batch)),
                                 dim3(kThreads), Ring<HD>::kBytes, s, static_cast<unsigned>(p.splits),
                                 a) == cudaSuccess
               ? SAL_OK
               : SAL_ECUDA;
  const unsigned grid = static_cast<unsigned>(p.grid);
  if (launch_kernel(paged_line_kernel<HD>, dim3(grid), dim3(kThreads), Ring<HD>::kBytes, s, a) != cudaSuccess)
    return SAL_ECUDA;
  if (a.inside) return SAL_OK;
  const int rows = std::min(kRowTile, a.heads / a.kv_heads);
  declare();
  const unsigned entries = a.by_part ? grid : static_cast<unsigned>(a.batch) * groups;
  return launch_kernel(paged_join_kernel<HD>, dim3(entries, static_cast<unsigned>(rows)), dim3(kJoinThreads), 0, s,
                       a) == cudaSuccess
             ? SAL_OK
             : SAL_ECUDA;
}

}  // namespace

size_t attention_paged_bytes(int head_dim) { return workspace_bytes(head_dim); }
size_t attention_paged_zero_bytes() { return kArrivedBytes; }

}  // namespace sal

extern "C" {

size_t sal_attention_paged_workspace_bytes(const sal_cache* cache, int batch, int heads) {
  using namespace sal;
  if (check_cache(cache, false) != SAL_OK || batch <= 0 || heads <= 0 || heads % cache->kv_heads != 0) return 0;
  return workspace_bytes(cache->head_dim);
}

sal_status sal_attention_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride, int batch, int heads,
                               const sal_cache* cache, int layer, const int32_t* seqs, const sal_window* window,
                               void* o, void* workspace, size_t ws_bytes, void* stream) {
  using namespace sal;
  const NvtxRange nvtx_("sal_attention_paged");
  const sal_status ok = check_cache(cache, false);
  if (ok != SAL_OK) return ok;
  if (batch < 0 || heads < 0 || layer < 0 || layer >= cache->layers) return SAL_EINVAL;
  if (q_row_stride < 0 || q_head_stride < 0 || (q_row_stride & 7) || (q_head_stride & 7)) return SAL_EINVAL;
  if (window && window->sinks < 0) return SAL_EINVAL;
  if (batch > 65535 || heads > 65535) return SAL_ESHAPE;
  if (batch == 0 || heads == 0) return SAL_OK;
  if (heads % cache->kv_heads != 0 || (!seqs && batch > cache->sequences)) return SAL_EINVAL;
  if (!q || !o || !aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(seqs) & 3u)) return SAL_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SAL_EINVAL;
  const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  const int64_t left = !window || window->left < 0 ? cap : std::min(window->left, cap);
  const int64_t sinks = window ? std::min(window->sinks, cap) : 0;
  const Plan plan = plan_of(cache, batch, heads, std::min(cap, left + 1 + sinks));
  if (ws_bytes < sal_attention_paged_workspace_bytes(cache, batch, heads)) return SAL_EWORKSPACE;
  if (static_cast<int64_t>(cache->kv_heads) * plan.row_tiles > 65535) return SAL_ESHAPE;
  sal_status st = require_device();
  if (st == SAL_OK) st = kernel_attributes();
  if (st != SAL_OK) return st;
  const int hd = cache->head_dim;
  const int64_t slab = static_cast<int64_t>(cache->pages) * cache->kv_heads * cache->page_size * hd;
  PagedArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(cache->k) + layer * slab;
  a.v = static_cast<const __nv_bfloat16*>(cache->v) + layer * slab;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.table = cache->table;
  a.lengths = cache->lengths;
  a.seqs = seqs;
  a.heads = heads;
  a.kv_heads = cache->kv_heads;
  a.pages = cache->pages;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(cache->page_size));
  a.sequences = cache->sequences;
  a.max_pages = cache->max_pages;
  a.left = static_cast<int>(left);
  a.sinks = static_cast<int>(sinks);
  a.row_tiles = plan.row_tiles;
  a.splits = plan.splits;
  a.by_part = static_cast<int64_t>(batch) * cache->kv_heads * plan.row_tiles > plan.grid;
  a.batch = batch;
  char* w = static_cast<char*>(workspace);
  a.arrived = reinterpret_cast<int*>(w);
  a.joins = reinterpret_cast<int4*>(w + kArrivedBytes);
  a.stats = reinterpret_cast<float2*>(w + kArrivedBytes + kJoinBytes);
  a.part = reinterpret_cast<float*>(w + kArrivedBytes + kJoinBytes + kStatBytes);
  // One thread owns a column of a row and reads its pieces one after the other: worth it for few of
  // both (64 rows with 10 heads: as fast, 49.4 us for 49.6, and one launch fewer, 2.3 us of the host's
  // time); many heads to a piece or pieces to a row go to a kernel with a block per row (3 rows of
  // 45,000 keys, 16 heads to a key head: 30.2 us, inside 47.7).
  const int64_t pairs = static_cast<int64_t>(batch) * cache->kv_heads * plan.row_tiles;
  a.inside = heads / cache->kv_heads <= 4 && pairs >= 32;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
  const auto declare = [&] {
    ck_declare(q, ((batch - 1) * q_row_stride + (heads - 1) * q_head_stride + hd) * 2, false);
    ck_declare(a.k, slab * 2, false);
    ck_declare(a.v, slab * 2, false);
    ck_declare(o, static_cast<uint64_t>(batch) * heads * hd * 2, true);
    ck_declare(a.table, static_cast<uint64_t>(a.sequences) * a.max_pages * 4, false);
    ck_declare(a.lengths, static_cast<uint64_t>(a.sequences) * 4, false);
    ck_declare(seqs, static_cast<uint64_t>(batch) * 4, false);
    ck_declare(workspace, workspace_bytes(hd), true);
  };
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return hd == 128 ? launch<128>(a, plan, s, declare) : launch<64>(a, plan, s, declare);
}

}  // extern "C"
