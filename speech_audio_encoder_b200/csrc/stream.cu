// The encoder's layers over live streams (sal_stream_prefill, sal_stream_step): the layer of
// sal_encoder_forward with causal windowed attention, its keys and values kept in a paged cache.
//
// A prefill is whole clips from position 0, so its QKV projection is the encoder's (QK-norm and
// RoPE in the epilogue); the windowed attention reads the rows it wrote and the cache gets a copy.
// A step has one row per stream, each at a position of its own: the projection writes fp32 rows,
// and one kernel normalises and rotates q and k (one warp per row and head, the lanes hold the
// rotate-half pairs l, l + 64 and l + 32, l + 96) and puts k and v straight into their pages. Its
// rotations come from a table that is built once a step, in 64 bits, since a stream's position
// times the fastest frequency needs more than the 24 bits of fp32.
//
// Both write at the lengths that the resize before them left on the device. One that failed has
// left the old lengths, and the newest position, whose page a fork may share, would be written
// over: so while the cache's status word is set neither keeps anything.
#define SAL_CK_FILE 9
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "sal_internal.h"
#include "sal_ptx.cuh"

namespace sal {
namespace {

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct StreamWs {
  void *h, *q, *k, *v, *o, *u;  // bf16: [M, 1280] each, u [M, 5120] over q, k, v and o
  float *qkv, *rope;            // step: [M, 3840]; prefill: [2, T, 64], step: [2, M, 64]
  void* paged;                  // step: scratch of the attention over the cache
  size_t bytes;
};

StreamWs layout(void* base, int batch, int64_t T) {
  const size_t M = static_cast<size_t>(batch) * static_cast<size_t>(T), act = align256(M * kWidth * 2);
  char* p = static_cast<char*>(base);
  StreamWs w{};
  size_t off = 0;
  auto take = [&](size_t n) {
    char* r = p + off;
    off += align256(n);
    return r;
  };
  w.h = take(act);
  char* big = take(std::max(4 * act, align256(M * kFfn * 2)));
  w.q = big;
  w.k = big + act;
  w.v = big + 2 * act;
  w.o = big + 3 * act;
  w.u = big;
  w.rope = reinterpret_cast<float*>(take(static_cast<size_t>(std::max<int64_t>(T, batch)) * 64 * 2 * 4));
  if (T == 1) {
    w.qkv = reinterpret_cast<float*>(take(M * 3 * kWidth * 4));
    w.paged = take(attention_paged_bytes(kHeadDim));
  }
  w.bytes = off;
  return w;
}

struct StepArgs {
  const float* qkv;
  const __nv_bfloat16 *qn_g, *kn_g;
  float* rope;  // [2][batch][64]
  __nv_bfloat16 *q, *k_pages, *v_pages;
  const int32_t *table, *lengths, *seqs;
  const uint32_t* failed;  // the cache's status word
  int batch, pages, page_shift, sequences, max_pages;
};

// The position of a row's new token, or -1 where there is none.
__device__ __forceinline__ int position_of(const StepArgs& a, int b, int& seq) {
  seq = a.seqs ? *SAL_CK_LD(a.seqs + b, 4) : b;
  if (seq < 0 || seq >= a.sequences) return -1;
  return min(max(*SAL_CK_LD(a.lengths + seq, 4), 0), a.max_pages << a.page_shift) - 1;
}

__global__ void __launch_bounds__(256) step_rope_kernel(const StepArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (i >= a.batch * 64) return;
  int seq;
  const int p = max(position_of(a, i >> 6, seq), 0);
  double s, c;
  sincos(p * pow(10000.0, -static_cast<double>(2 * (i & 63)) / 128.0), &s, &c);
  *SAL_CK_ST(a.rope + i, 4) = static_cast<float>(c);
  *SAL_CK_ST(a.rope + a.batch * 64 + i, 4) = static_cast<float>(s);
}

__global__ void __launch_bounds__(256) step_qkv_kernel(const StepArgs a) {
  const int lane = threadIdx.x & 31, unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (unit >= a.batch * kHeads) return;
  const int b = unit / kHeads, h = unit - b * kHeads;
  const float* src = a.qkv + static_cast<int64_t>(b) * (3 * kWidth) + h * kHeadDim;
  float c[2], s[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = *SAL_CK_LD(a.rope + b * 64 + lane + 32 * e, 4);
    s[e] = *SAL_CK_LD(a.rope + (a.batch + b) * 64 + lane + 32 * e, 4);
  }
  // x[e] and x[e + 2] are the pair of angle lane + 32 e
  auto rotated = [&](const float* x0, const __nv_bfloat16* gain, float (&x)[4]) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = *SAL_CK_LD(x0 + lane + 32 * e, 4);
      sq += x[e] * x[e];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
    const float r = rsqrtf(sq * (1.0f / kHeadDim) + 1e-6f);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= r * __bfloat162float(*SAL_CK_LD(gain + lane + 32 * e, 2));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float lo = x[e] * c[e] - x[e + 2] * s[e], hi = x[e + 2] * c[e] + x[e] * s[e];
      x[e] = lo;
      x[e + 2] = hi;
    }
  };
  float x[4];
  rotated(src, a.qn_g, x);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *SAL_CK_ST(a.q + static_cast<int64_t>(unit) * kHeadDim + lane + 32 * e, 2) = __float2bfloat16(x[e]);
  int seq;
  const int p = position_of(a, b, seq);
  if (p < 0 || *SAL_CK_LD(a.failed, 4)) return;
  const int page = *SAL_CK_LD(a.table + static_cast<int64_t>(seq) * a.max_pages + (p >> a.page_shift), 4);
  if (page < 0 || page >= a.pages) return;
  const int64_t at = (((static_cast<int64_t>(page) * kHeads + h) << a.page_shift) + (p & ((1 << a.page_shift) - 1))) *
                     kHeadDim + lane;
  rotated(src + kWidth, a.kn_g, x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    *SAL_CK_ST(a.k_pages + at + 32 * e, 2) = __float2bfloat16(x[e]);
    *SAL_CK_ST(a.v_pages + at + 32 * e, 2) = __float2bfloat16(*SAL_CK_LD(src + 2 * kWidth + lane + 32 * e, 4));
  }
}

// The checks that both calls share.
sal_status check_call(const float* x, int batch, int64_t T, const sal_weights* w, int n_layers, const sal_window* window,
                      const sal_cache* cache, const int32_t* seqs, const void* emb, const void* workspace) {
  const sal_status st = check_cache(cache, false);
  if (st != SAL_OK) return st;
  if (batch < 0 || T < 0 || !w || n_layers < 0 || n_layers > w->n_layers || (window && window->sinks < 0))
    return SAL_EINVAL;
  if (T > SAL_MAX_POSITIONS || batch > 6553) return SAL_ESHAPE;
  if (cache->kv_heads != kHeads || cache->head_dim != kHeadDim || cache->layers < n_layers) return SAL_ESHAPE;
  if (!seqs && batch > cache->sequences) return SAL_EINVAL;
  if (batch == 0 || T == 0) return SAL_OK;
  if (!x || !emb || !aligned16(x) || !aligned16(emb) || (reinterpret_cast<uintptr_t>(seqs) & 3u)) return SAL_EINVAL;
  if (!w->lnf_g || !w->lnf_b || !aligned16(w->lnf_g) || !aligned16(w->lnf_b)) return SAL_EINVAL;
  if (n_layers > 0 && !w->layers) return SAL_EINVAL;
  for (int i = 0; i < n_layers; ++i)
    if (!layer_parameters_ok(w->layers[i])) return SAL_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SAL_EINVAL;
  return SAL_OK;
}

}  // namespace
}  // namespace sal

using namespace sal;

#define SAL_TRY(expr)              \
  do {                             \
    const sal_status st_ = (expr); \
    if (st_ != SAL_OK) return st_; \
  } while (0)

extern "C" {

size_t sal_stream_workspace_bytes(int batch, int64_t T) {
  if (batch <= 0 || T <= 0) return 0;
  return layout(nullptr, batch, T).bytes;
}

sal_status sal_stream_prefill(float* x, int batch, int64_t T, const int32_t* lengths, const sal_weights* w,
                              int n_layers, const sal_window* window, const sal_cache* cache, const int32_t* seqs,
                              void* emb, void* workspace, size_t ws_bytes, void* stream) {
  const NvtxRange nvtx_("sal_stream_prefill");
  SAL_TRY(check_call(x, batch, T, w, n_layers, window, cache, seqs, emb, workspace));
  if (reinterpret_cast<uintptr_t>(lengths) & 3u) return SAL_EINVAL;
  if (batch == 0 || T == 0) return SAL_OK;
  const StreamWs ws = layout(workspace, batch, T);
  if (ws_bytes < ws.bytes) return SAL_EWORKSPACE;
  SAL_TRY(require_device());
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t M = static_cast<int64_t>(batch) * T;
  const sal_window win{window ? window->left : -1, 0, window ? window->sinks : 0};
  if (n_layers > 0) SAL_TRY(rope_table_launch(ws.rope, T, s));
  for (int i = 0; i < n_layers; ++i) {
    const sal_layer& L = w->layers[i];
    SAL_TRY(layernorm_launch(x, M, L.ln1_g, L.ln1_b, ws.h, s));
    QkvOut qo{ws.q, ws.k, ws.v, L.qn_g, L.kn_g, ws.rope, T, 0};
    SAL_TRY(gemm_launch(kEpiQkv, ws.h, M, kWidth, L.w_qkv, 3 * kWidth, L.b_qkv, nullptr, &qo, s));
    SAL_TRY(cache_append(cache, i, ws.k, ws.v, batch, T, nullptr, seqs, true, s));
    SAL_TRY(window_attention_launch(ws.q, ws.k, ws.v, batch, T, kHeads, kHeads, kHeadDim, win, lengths, ws.o, s));
    SAL_TRY(gemm_launch(SAL_EPI_RESID_F32, ws.o, M, kWidth, L.w_o, kWidth, L.b_o, x, nullptr, s));
    SAL_TRY(layernorm_launch(x, M, L.ln2_g, L.ln2_b, ws.h, s));
    SAL_TRY(gemm_launch(SAL_EPI_GELU_BF16, ws.h, M, kWidth, L.w1, kFfn, L.b1, ws.u, nullptr, s));
    SAL_TRY(gemm_launch(SAL_EPI_RESID_F32, ws.u, M, kFfn, L.w2, kWidth, L.b2, x, nullptr, s));
  }
  return layernorm_launch(x, M, w->lnf_g, w->lnf_b, emb, s);
}

sal_status sal_stream_step(float* x, int batch, const sal_weights* w, int n_layers, const sal_window* window,
                           const sal_cache* cache, const int32_t* seqs, void* emb, void* workspace, size_t ws_bytes,
                           void* stream) {
  const NvtxRange nvtx_("sal_stream_step");
  SAL_TRY(check_call(x, batch, 1, w, n_layers, window, cache, seqs, emb, workspace));
  if (batch == 0) return SAL_OK;
  const StreamWs ws = layout(workspace, batch, 1);
  if (ws_bytes < ws.bytes) return SAL_EWORKSPACE;
  SAL_TRY(require_device());
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const sal_window win{window ? window->left : -1, 0, window ? window->sinks : 0};
  StepArgs a{};
  a.qkv = ws.qkv;
  a.rope = ws.rope;
  a.q = static_cast<__nv_bfloat16*>(ws.q);
  a.table = cache->table;
  a.lengths = cache->lengths;
  a.seqs = seqs;
  a.failed = cache->status;
  a.batch = batch;
  a.pages = cache->pages;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(cache->page_size));
  a.sequences = cache->sequences;
  a.max_pages = cache->max_pages;
  const int64_t slab = static_cast<int64_t>(cache->pages) * kHeads * cache->page_size * kHeadDim;
  const auto declare = [&] {
    ck_declare(a.table, static_cast<uint64_t>(a.sequences) * a.max_pages * 4, false);
    ck_declare(a.lengths, static_cast<uint64_t>(a.sequences) * 4, false);
    ck_declare(seqs, static_cast<uint64_t>(batch) * 4, false);
    ck_declare(a.rope, static_cast<uint64_t>(batch) * 64 * 2 * 4, true);
  };
  if (n_layers > 0) {
    if (cudaMemsetAsync(ws.paged, 0, attention_paged_zero_bytes(), s) != cudaSuccess) return SAL_ECUDA;
    declare();
    if (launch_kernel(step_rope_kernel, dim3(static_cast<unsigned>((batch * 64 + 255) / 256)), dim3(256), 0, s, a) !=
        cudaSuccess)
      return SAL_ECUDA;
  }
  for (int i = 0; i < n_layers; ++i) {
    const sal_layer& L = w->layers[i];
    SAL_TRY(layernorm_launch(x, batch, L.ln1_g, L.ln1_b, ws.h, s));
    SAL_TRY(gemm_launch(SAL_EPI_STORE_F32, ws.h, batch, kWidth, L.w_qkv, 3 * kWidth, L.b_qkv, ws.qkv, nullptr, s));
    a.qn_g = static_cast<const __nv_bfloat16*>(L.qn_g);
    a.kn_g = static_cast<const __nv_bfloat16*>(L.kn_g);
    a.k_pages = static_cast<__nv_bfloat16*>(cache->k) + i * slab;
    a.v_pages = static_cast<__nv_bfloat16*>(cache->v) + i * slab;
    declare();
    ck_declare(a.qkv, static_cast<uint64_t>(batch) * 3 * kWidth * 4, false);
    ck_declare(a.qn_g, kHeadDim * 2, false);
    ck_declare(a.kn_g, kHeadDim * 2, false);
    ck_declare(a.failed, 4, false);
    ck_declare(a.q, static_cast<uint64_t>(batch) * kWidth * 2, true);
    ck_declare(a.k_pages, static_cast<uint64_t>(slab) * 2, true);
    ck_declare(a.v_pages, static_cast<uint64_t>(slab) * 2, true);
    if (launch_kernel(step_qkv_kernel, dim3(static_cast<unsigned>((batch * kHeads + 7) / 8)), dim3(256), 0, s, a) !=
        cudaSuccess)
      return SAL_ECUDA;
    SAL_TRY(sal_attention_paged(ws.q, kWidth, kHeadDim, batch, kHeads, cache, i, seqs, &win, ws.o, ws.paged,
                                attention_paged_bytes(kHeadDim), stream));
    SAL_TRY(gemm_launch(SAL_EPI_RESID_F32, ws.o, batch, kWidth, L.w_o, kWidth, L.b_o, x, nullptr, s));
    SAL_TRY(layernorm_launch(x, batch, L.ln2_g, L.ln2_b, ws.h, s));
    SAL_TRY(gemm_launch(SAL_EPI_GELU_BF16, ws.h, batch, kWidth, L.w1, kFfn, L.b1, ws.u, nullptr, s));
    SAL_TRY(gemm_launch(SAL_EPI_RESID_F32, ws.u, batch, kFfn, L.w2, kWidth, L.b2, x, nullptr, s));
  }
  return layernorm_launch(x, batch, w->lnf_g, w->lnf_b, emb, s);
}

}  // extern "C"
