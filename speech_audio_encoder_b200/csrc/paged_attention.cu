// Attention of one new position per sequence over a paged key/value cache (sal_attention_paged):
// row b's query is position p = n - 1 of its sequence of n positions, and
//   o[b, h, :] = sum_j a_j v_j,  a = softmax_j(q k_j / sqrt(d)) over the keys j < n with
//   j >= p - left or j < sinks, whose page the table still names.
// One warp per (row, head), lanes across the head dimension.
#define SAL_CK_FILE 7
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "sal_internal.h"
#include "sal_ptx.cuh"

namespace sal {
namespace {

struct PagedArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  int64_t q_row, q_head;
  const int32_t *table, *lengths, *seqs;
  int batch, heads, kv_heads, pages, page_shift, sequences, max_pages;
  int left, sinks;
};

template <int HD>
__global__ void __launch_bounds__(256) paged_simple_kernel(const PagedArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (row >= static_cast<int64_t>(a.batch) * a.heads) return;
  const int h = static_cast<int>(row % a.heads), b = static_cast<int>(row / a.heads);
  const int seq = a.seqs ? *SAL_CK_LD(a.seqs + b, 4) : b;
  int n = 0;
  if (seq >= 0 && seq < a.sequences) n = min(max(*SAL_CK_LD(a.lengths + seq, 4), 0), a.max_pages << a.page_shift);
  const int kvh = h / (a.heads / a.kv_heads), lo = max(0, n - 1 - a.left), s = min(a.sinks, lo);
  const float scale = 1.0f / sqrtf(static_cast<float>(HD));
  float qv[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(*SAL_CK_LD(a.q + b * a.q_row + h * a.q_head + e * 32 + lane, 2)) * scale;
    acc[e] = 0.f;
  }
  for (int i = 0; i < s + n - lo; ++i) {
    const int j = i < s ? i : lo + i - s;
    const int page = *SAL_CK_LD(a.table + static_cast<int64_t>(seq) * a.max_pages + (j >> a.page_shift), 4);
    if (page < 0 || page >= a.pages) continue;
    const int64_t at = (((static_cast<int64_t>(page) * a.kv_heads + kvh) << a.page_shift) +
                        (j & ((1 << a.page_shift) - 1))) * HD + lane;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += qv[e] * __bfloat162float(*SAL_CK_LD(a.k + at + e * 32, 2));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float mn = fmaxf(m, x), f = expf(m - mn), w = expf(x - mn);
    l = l * f + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * __bfloat162float(*SAL_CK_LD(a.v + at + e * 32, 2));
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    *SAL_CK_ST(a.o + row * HD + e * 32 + lane, 2) = __float2bfloat16(l > 0.f ? acc[e] / l : 0.f);
}

}  // namespace
}  // namespace sal

extern "C" {

size_t sal_attention_paged_workspace_bytes(const sal_cache* cache, int batch, int heads) {
  if (!cache || batch <= 0 || heads <= 0) return 0;
  return 256;
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
  if (ws_bytes < sal_attention_paged_workspace_bytes(cache, batch, heads)) return SAL_EWORKSPACE;
  const sal_status st = require_device();
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
  a.batch = batch;
  a.heads = heads;
  a.kv_heads = cache->kv_heads;
  a.pages = cache->pages;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(cache->page_size));
  a.sequences = cache->sequences;
  a.max_pages = cache->max_pages;
  const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  a.left = static_cast<int>(!window || window->left < 0 ? cap : std::min<int64_t>(window->left, cap));
  a.sinks = static_cast<int>(window ? std::min<int64_t>(window->sinks, cap) : 0);
  ck_declare(q, ((batch - 1) * q_row_stride + (heads - 1) * q_head_stride + hd) * 2, false);
  ck_declare(a.k, slab * 2, false);
  ck_declare(a.v, slab * 2, false);
  ck_declare(o, static_cast<uint64_t>(batch) * heads * hd * 2, true);
  ck_declare(a.table, static_cast<uint64_t>(a.sequences) * a.max_pages * 4, false);
  ck_declare(a.lengths, static_cast<uint64_t>(a.sequences) * 4, false);
  ck_declare(seqs, static_cast<uint64_t>(batch) * 4, false);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(batch) * heads + 7) / 8));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = hd == 128 ? launch_kernel(paged_simple_kernel<128>, grid, dim3(256), 0, s, a)
                                  : launch_kernel(paged_simple_kernel<64>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? SAL_OK : SAL_ECUDA;
}

}  // extern "C"
