// Attention with a sliding window and first positions that stay visible (sal_attention_window):
//   o[b, p, h, :] = sum_j a_pj v_j,  a = softmax_j(q_p k_j / sqrt(d)) over the keys j < n_b with
//   j <= p + right and (j >= p - left or j < sinks).
// One warp per (clip, head, position): the lanes hold the row's q and its accumulator, each
// key is one warp sum, the maximum and sum of the softmax run along.
#define SAL_CK_FILE 6
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "sal_internal.h"
#include "sal_ptx.cuh"

namespace sal {
namespace {

struct WindowArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  const int32_t* lengths;
  int batch, T, heads, kv_heads;
  int left, right, sinks;
};

template <int HD>
__global__ void __launch_bounds__(256) window_simple_kernel(const WindowArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (row >= static_cast<int64_t>(a.batch) * a.heads * a.T) return;
  const int p = static_cast<int>(row % a.T);
  const int h = static_cast<int>(row / a.T % a.heads), b = static_cast<int>(row / a.T / a.heads);
  const int n = a.lengths ? min(max(*SAL_CK_LD(a.lengths + b, 4), 0), a.T) : a.T;
  if (p >= n) return;
  const int64_t kv = (static_cast<int64_t>(b) * a.kv_heads + h / (a.heads / a.kv_heads)) * a.T;
  const int lo = max(0, p - a.left), hi = min(n, p + a.right + 1), s = min(min(a.sinks, lo), hi);
  const float scale = 1.0f / sqrtf(static_cast<float>(HD));
  float qv[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(*SAL_CK_LD(a.q + row * HD + e * 32 + lane, 2)) * scale;
    acc[e] = 0.f;
  }
  for (int i = 0; i < s + hi - lo; ++i) {
    const int64_t j = i < s ? i : lo + i - s;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += qv[e] * __bfloat162float(*SAL_CK_LD(a.k + (kv + j) * HD + e * 32 + lane, 2));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float mn = fmaxf(m, x), f = expf(m - mn), w = expf(x - mn);
    l = l * f + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = acc[e] * f + w * __bfloat162float(*SAL_CK_LD(a.v + (kv + j) * HD + e * 32 + lane, 2));
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    *SAL_CK_ST(a.o + ((static_cast<int64_t>(b) * a.T + p) * a.heads + h) * HD + e * 32 + lane, 2) =
        __float2bfloat16(acc[e] / l);
}

}  // namespace

sal_status window_attention_launch(const void* q, const void* k, const void* v, int batch, int64_t T, int heads,
                                   int kv_heads, int head_dim, const sal_window& win, const int32_t* lengths, void* o,
                                   cudaStream_t s) {
  WindowArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lengths = lengths;
  a.batch = batch;
  a.T = static_cast<int>(T);
  a.heads = heads;
  a.kv_heads = kv_heads;
  // no limit and any limit past the clip are the same; all sums of these stay in 32 bits
  a.left = win.left < 0 ? a.T : static_cast<int>(std::min<int64_t>(win.left, T));
  a.right = win.right < 0 ? a.T : static_cast<int>(std::min<int64_t>(win.right, T));
  a.sinks = static_cast<int>(std::min<int64_t>(win.sinks, T));
  const int64_t rows = static_cast<int64_t>(batch) * heads * T;
  ck_declare(q, rows * head_dim * 2, false);
  ck_declare(k, static_cast<int64_t>(batch) * kv_heads * T * head_dim * 2, false);
  ck_declare(v, static_cast<int64_t>(batch) * kv_heads * T * head_dim * 2, false);
  ck_declare(o, rows * head_dim * 2, true);
  ck_declare(lengths, static_cast<uint64_t>(batch) * 4, false);
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
  const cudaError_t e = head_dim == 128 ? launch_kernel(window_simple_kernel<128>, grid, dim3(256), 0, s, a)
                                        : launch_kernel(window_simple_kernel<64>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? SAL_OK : SAL_ECUDA;
}

}  // namespace sal

extern "C" sal_status sal_attention_window(const void* q, const void* k, const void* v, int batch, int64_t T,
                                           int heads, int kv_heads, int head_dim, const sal_window* window,
                                           const int32_t* lengths, void* o, void* stream) {
  using namespace sal;
  const NvtxRange nvtx_("sal_attention_window");
  if (batch < 0 || T < 0 || heads < 0 || kv_heads < 0) return SAL_EINVAL;
  if (window && window->sinks < 0) return SAL_EINVAL;
  if (head_dim != 64 && head_dim != 128) return SAL_ESHAPE;
  if (T > 2 * SAL_MAX_POSITIONS) return SAL_ESHAPE;
  if (batch == 0 || T == 0 || heads == 0) return SAL_OK;
  if (kv_heads == 0 || heads % kv_heads != 0) return SAL_EINVAL;
  if (static_cast<int64_t>(batch) * heads > 65535) return SAL_ESHAPE;
  if (!q || !k || !v || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return SAL_EINVAL;
  const sal_status st = require_device();
  if (st != SAL_OK) return st;
  const sal_window all{-1, -1, 0};
  return window_attention_launch(q, k, v, batch, T, heads, kv_heads, head_dim, window ? *window : all, lengths, o,
                                 static_cast<cudaStream_t>(stream));
}
