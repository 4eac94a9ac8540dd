// Attention with a sliding window and first positions that stay visible (sal_attention_window):
//   o[b, p, h, :] = sum_j a_pj v_j,  a = softmax_j(q_p k_j / sqrt(d)) over the keys j < n_b with
//   j <= p + right and (j >= p - left or j < sinks).
//
// One pass over the visible keys with the running maximum and sum of the softmax, on the tensor
// cores: a tile of 128 query rows takes only the 128-key tiles its rows can see - those of the
// first positions, then those of the window - and masks single scores only in tiles that a
// limit cuts. A block holds two query tiles ("slots") that share every key tile it loads: two
// query heads of one key head where heads come in such pairs (both see the same tiles), else two
// neighbouring tiles of one head (a tile that only one of them sees is skipped by the other).
// The tensor core reads 64 KB of K and V for 4 * 128 * 128 * 128 flops of one slot; without
// the second slot the loads from L2 would bound it.
//
// Windows are short (a minute is six tiles), so starting and ending would cost as much as the
// work: the blocks are persistent, one per SM, and every role runs ahead into the next work item
// as far as its buffers allow - the next Q and K are loaded while the last products run, and
// one slot stores its rows while the other still multiplies.
//
// Roles: warp 0 loads (TMA); warp 1 issues S_i = Q_i K^T; warp 2 issues O_i += P_i V; warps 4-7 and
// 8-11 are the softmax of slot 0 and 1, one row per thread. TMEM: at head dim 128 one score
// buffer S [0,128) that the slots take in turn (a slot copies its scores to registers and hands
// it back), O0 [128,256) O1 [256,384) P0 [384,448) P1 [448,512); at 64 a buffer each: S0 [0,128)
// S1 [128,256) O0 [256,320) O1 [320,384), P as above. P is rounded to bf16 for its product
// (the row sum is not); scores, maxima, sums and O are fp32.
#define SAL_CK_FILE 6
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "sal_internal.h"
#include "sal_ptx.cuh"

namespace sal {
namespace {

constexpr int kTile = 128;
constexpr int kBox = kTile * 64 * 2;       // one 64-column half of a 128 x 128 bf16 tile
constexpr float kRescaleThreshold = 8.0f;  // log2 units: below it the old maximum stays (p <= 256)
constexpr int kThreads = 384;
constexpr int kRegsCtrl = 104, kRegsSoftmax = 200;
constexpr int kRegsNeeded = kRegsCtrl * 128 + kRegsSoftmax * 256;  // <= launch registers x 384
constexpr int kLengths = 512;  // clip lengths kept in shared memory

template <int HD>
struct Layout {
  static constexpr int kTileB = kTile * HD * 2;  // a 128-row tile of Q, K or V
  static constexpr int kBoxes = HD / 64;         // 64-column boxes of a tile
  static constexpr bool kSharedS = HD == 128;
  static constexpr int kStages = 2;
  static constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * static_cast<size_t>(kTileB) + 512 + 4 * kLengths;
  __device__ static uint32_t col_s(int i) { return kSharedS ? 0u : 128u * i; }
  __device__ static uint32_t col_o(int i) { return kSharedS ? 128u + 128u * i : 256u + 64u * i; }
  __device__ static uint32_t col_p(int i) { return 384u + 64u * i; }
};
static_assert(Layout<128>::kSmem <= 227 * 1024 && Layout<64>::kSmem <= 227 * 1024, "shared memory");

enum Pairing { kSingles, kTilePairs, kHeadPairs };

struct WindowArgs {
  __nv_bfloat16* o;
  const int32_t* lengths;
  int batch, T, heads, kv_heads;
  int left, right, sinks;  // left, right: T for no limit
  int tiles;               // query tiles of a clip
  int pairing, items;
  float scale_log2;
  uint64_t limit_ns;
  unsigned int* status;
};

// One work item: up to two query tiles and the key tiles they share. Key tile x of the item is
// tile(x) of the clip: x < first are those of the first positions, then the window's.
struct Item {
  int b, n, kv;               // clip, its length, its (clip, key head) plane
  int head[2], row[2];        // query head and first row of each slot
  int lo[2], hi[2], sink[2];  // a slot's window tiles [lo, hi) and first-position tiles [0, sink); hi = 0: empty
  int first, w0, count;
  __device__ int tile(int x) const { return x < first ? x : w0 + (x - first); }
  __device__ bool uses(int i, int x) const {
    const int t = tile(x);
    return t < hi[i] && (t >= lo[i] || t < sink[i]);
  }
  __device__ int last(int i) const { return first + hi[i] - 1 - w0; }  // the slot's last x
};

__device__ __forceinline__ Item item_of(const WindowArgs& a, int idx, const int* lens) {
  Item it;
  // the rows of the longest reach (a causal clip's last tiles) come first
  int h, t0;
  if (a.pairing == kHeadPairs) {
    const int planes = a.batch * (a.heads >> 1), pl = idx % planes;
    it.b = pl / (a.heads >> 1);
    h = 2 * (pl % (a.heads >> 1));
    t0 = a.tiles - 1 - idx / planes;
  } else {
    const int planes = a.batch * a.heads, pl = idx % planes;
    it.b = pl / a.heads;
    h = pl % a.heads;
    t0 = a.pairing == kTilePairs ? 2 * ((a.tiles + 1) / 2 - 1 - idx / planes) : a.tiles - 1 - idx / planes;
  }
  it.n = a.T;
  if (a.lengths) it.n = min(max(it.b < kLengths ? lens[it.b] : *SAL_CK_LD(a.lengths + it.b, 4), 0), a.T);
  it.kv = it.b * a.kv_heads + h / (a.heads / a.kv_heads);
  it.w0 = 1 << 30;
  int w1 = 0, sinks = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    it.head[i] = h + (a.pairing == kHeadPairs ? i : 0);
    it.row[i] = kTile * (t0 + (a.pairing == kTilePairs ? i : 0));
    it.lo[i] = it.hi[i] = it.sink[i] = 0;
    if (it.row[i] >= it.n || (i == 1 && a.pairing == kSingles)) continue;
    const int end = min(it.n, min(it.row[i] + kTile, it.n) + a.right);  // keys below it are in reach
    it.lo[i] = max(0, it.row[i] - a.left) / kTile;
    it.hi[i] = (end + kTile - 1) / kTile;
    it.sink[i] = (min(a.sinks, end) + kTile - 1) / kTile;
    it.w0 = min(it.w0, it.lo[i]);
    w1 = max(w1, it.hi[i]);
    sinks = max(sinks, it.sink[i]);
  }
  it.first = min(it.w0, sinks);
  it.count = w1 > 0 ? it.first + w1 - it.w0 : 0;
  return it;
}

// Maximum of a row of 128 scores held as raw fp32 bits, in eight independent chains.
__device__ __forceinline__ float row_max128(const uint32_t (&r)[4][32]) {
  float m[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t* v = &r[k >> 1][(k & 1) * 16];
    m[k] = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
    for (int i = 2; i < 16; i += 2) m[k] = max3f(m[k], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
  }
  return max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

// Bits [lo, hi) of a 32-bit word (both clamped to it).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
  const uint32_t below_lo = lo == 32 ? 0xffffffffu : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const WindowArgs args) {
  using L = Layout<HD>;
  constexpr int TB = L::kTileB, NS = L::kStages;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                // Q0, Q1
  uint8_t* sK = smem + 2 * TB;       // [NS]
  uint8_t* sV = sK + NS * TB;        // [NS]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NS * TB);
  uint64_t* q_full = bars;           // [2] Q_i has landed
  uint64_t* q_empty = bars + 2;      // [2] the item's last S_i has read Q_i
  uint64_t* s_full = bars + 4;       // [2] S_i is in its buffer
  uint64_t* s_free = bars + 6;       // [2] a buffer has been read ([0] alone where it is shared)
  uint64_t* p_full = bars + 8;       // [2] P_i is stored and O_i rescaled
  uint64_t* pv_done = bars + 10;     // [2] P_i V is in O_i
  uint64_t* drains = bars + 12;      // [2] wind-down of the issuers
  uint64_t* k_full = bars + 14;      // [NS]
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_full + 2 * NS;
  uint64_t* v_empty = k_full + 3 * NS;
  volatile int* s_issued = reinterpret_cast<volatile int*>(k_full + 4 * NS);  // [2] S products issued per slot
  volatile int* abort_flag = s_issued + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(s_issued) + 3);
  int* lens = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
  static_assert((14 + 4 * NS) * 8 + 16 <= 512, "barriers");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);  // one arrival per warp of the slot that read it
      mbar_init(&p_full[i], 128);
      mbar_init(&pv_done[i], 1);
      mbar_init(&drains[i], 1);
      s_issued[i] = 0;
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (args.lengths)
    for (int i = threadIdx.x; i < min(args.batch, kLengths); i += kThreads) lens[i] = *SAL_CK_LD(args.lengths + i, 4);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitGuard guard{abort_flag, args.limit_ns, args.status};
  // the producer's record of what it has loaded, for the wind-down
  uint32_t loads_q[2] = {0, 0}, loads_k = 0, loads_v = 0;
  bool ok = true;
  // Each role runs inside the branch that set its register limit.
  if (warp < 4) {
    setmaxnreg_dec<kRegsCtrl>();
    if (warp == 0 && lane == 0) {
      for (int idx = blockIdx.x; ok && idx < args.items; idx += gridDim.x) {
        const Item it = item_of(args, idx, lens);
        for (int x = 0; ok && x < it.count; ++x) {
          const uint32_t s = loads_k % NS, par = (loads_k / NS) & 1;
          const int row = it.tile(x) * kTile;
          if (!(ok = mbar_wait(&k_empty[s], par ^ 1, guard))) break;
          mbar_arrive_expect_tx(&k_full[s], TB);
          for (int b = 0; b < L::kBoxes; ++b) tma_load_3d(sK + s * TB + b * kBox, &tmK, &k_full[s], 64 * b, row, it.kv);
          ++loads_k;
          // an item's queries behind its first key tile, which the ring could take earlier
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (x > 0 || !ok || it.hi[i] == 0) continue;
            if (!(ok = mbar_wait(&q_empty[i], (loads_q[i] & 1) ^ 1, guard))) continue;
            mbar_arrive_expect_tx(&q_full[i], TB);
            for (int b = 0; b < L::kBoxes; ++b)
              tma_load_3d(sQ + i * TB + b * kBox, &tmQ, &q_full[i], 64 * b, it.row[i], it.b * args.heads + it.head[i]);
            ++loads_q[i];
          }
          if (!ok || !(ok = mbar_wait(&v_empty[s], par ^ 1, guard))) break;
          mbar_arrive_expect_tx(&v_full[s], TB);
          for (int b = 0; b < L::kBoxes; ++b) tma_load_3d(sV + s * TB + b * kBox, &tmV, &v_full[s], 64 * b, row, it.kv);
          ++loads_v;
        }
      }
    } else if (warp == 1 && lane == 0) {
      constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
      uint32_t n_k = 0, n_s[2] = {0, 0}, n_q[2] = {0, 0};
      for (int idx = blockIdx.x; ok && idx < args.items; idx += gridDim.x) {
        const Item it = item_of(args, idx, lens);
        bool begun[2] = {false, false};
        for (int x = 0; ok && x < it.count; ++x) {
          const uint32_t s = n_k % NS;
          if (!(ok = mbar_wait(&k_full[s], (n_k / NS) & 1, guard))) break;
          ++n_k;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || !it.uses(i, x)) continue;
            if (!begun[i]) {
              if (!(ok = mbar_wait(&q_full[i], n_q[i] & 1, guard))) continue;
              ++n_q[i];
              begun[i] = true;
            }
            // the buffer's last scores have been read out of it
            const uint32_t before = L::kSharedS ? n_s[0] + n_s[1] : n_s[i];
            if (before > 0 && !(ok = mbar_wait(&s_free[L::kSharedS ? 0 : i], (before - 1) & 1, guard)))
              continue;
            tc_fence_after();
            const uint32_t q0 = smem_u32(sQ + i * TB), k0 = smem_u32(sK + s * TB);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
              umma_ss(tmem + L::col_s(i), sdesc_kmajor_sw128(q0 + off), sdesc_kmajor_sw128(k0 + off), IDESC_S, kk > 0);
            }
            umma_commit(&s_full[i]);
            s_issued[i] = ++n_s[i];
            if (x == it.last(i)) umma_commit(&q_empty[i]);
          }
          if (ok) umma_commit(&k_empty[s]);
        }
      }
      if (*abort_flag) {
        umma_commit(&drains[0]);
        drain_wait(&drains[0], 0);
      }
    } else if (warp == 2) {
      constexpr uint32_t IDESC_O = idesc_bf16(128, HD, false, true);
      uint32_t n_v = 0, n_p[2] = {0, 0};
      for (int idx = blockIdx.x; ok && idx < args.items; idx += gridDim.x) {
        const Item it = item_of(args, idx, lens);
        bool begun[2] = {false, false};
        for (int x = 0; ok && x < it.count; ++x) {
          const uint32_t s = n_v % NS;
          if (lane == 0) ok = mbar_wait(&v_full[s], (n_v / NS) & 1, guard);
          if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
          ++n_v;
          const int base = it.tile(x) * kTile;
          if (base + kTile > it.n && it.n < args.T) {
            // rows past the clip's length hold anything (NaN times a weight of zero is NaN): zeros
            __syncwarp();
            for (int r = it.n - base + (lane >> 3); r < kTile; r += 4)
              for (int b = 0; b < L::kBoxes; ++b)
                *reinterpret_cast<uint4*>(sV + s * TB + b * kBox + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || !it.uses(i, x)) continue;
              if (!(ok = mbar_wait(&p_full[i], n_p[i] & 1, guard))) continue;
              if (x != it.last(i)) {
                // the tensor core runs products in the order they are issued: the slot's next S, which
                // its softmax waits for, goes ahead of this product. A short spin, its bound checked
                // every 64 polls.
                const int need = static_cast<int>(n_p[i]) + 2;
                uint64_t t0 = 0;
                for (uint32_t spin = 1; s_issued[i] < need; ++spin) {
                  if ((spin & 63) != 0) continue;
                  if (*abort_flag) {
                    ok = false;
                    break;
                  }
                  const uint64_t now = globaltimer_ns();
                  if (t0 == 0) {
                    t0 = now;
                  } else if (now - t0 > args.limit_ns) {
                    *abort_flag = 1;
                    atomicOr(args.status, kStatusTimeout);
                    ok = false;
                    break;
                  }
                }
                if (!ok) continue;
              }
              tc_fence_after();
              const uint32_t v0 = smem_u32(sV + s * TB);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_ts(tmem + L::col_o(i), tmem + L::col_p(i) + kk * 8, sdesc_mnmajor_sw128(v0 + kk * 2048, kBox),
                        IDESC_O, (begun[i] || kk > 0));
              umma_commit(&pv_done[i]);
              begun[i] = true;
              ++n_p[i];
            }
            if (ok) umma_commit(&v_empty[s]);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      if (lane == 0 && *abort_flag) {
        umma_commit(&drains[1]);
        drain_wait(&drains[1], 0);
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    const int wg = (warp - 4) >> 2;  // slot
    const int quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t colS = L::col_s(wg), colO = L::col_o(wg), colP = L::col_p(wg);
    const int row = quarter * 32 + lane;
    const float sl2 = args.scale_log2;
    uint32_t n_s = 0;  // score tiles of this slot so far
    for (int idx = blockIdx.x; ok && idx < args.items; idx += gridDim.x) {
      const Item it = item_of(args, idx, lens);
      if (it.hi[wg] == 0) continue;
      const int p = it.row[wg] + row;
      const int key_lo = max(0, p - args.left), key_hi = min(it.n, p + args.right + 1), key_sink = min(args.sinks, key_hi);
      float m_ref = -INFINITY, l = 0.f;
      bool begun = false;
      for (int x = 0; x < it.count; ++x) {
        if (!it.uses(wg, x)) continue;
        if (!(ok = mbar_wait_warp(&s_full[wg], n_s & 1, guard))) break;
        tc_fence_after();
        // the whole row of scores in registers, then the buffer goes back to the tensor core
        uint32_t r[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_base + colS + 32 * c, r[c]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[L::kSharedS ? 0 : wg]);
        const int base = it.tile(x) * kTile;
        const int c_hi = key_hi - base, c_sink = key_sink - base;
        const int c_lo = c_sink >= key_lo - base ? 0 : key_lo - base;  // first positions that reach the window
        if (!__all_sync(0xffffffffu, c_hi >= kTile && c_lo <= 0)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = bits_between(c_lo - 32 * c, c_hi - 32 * c) | bits_between(0, c_sink - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1u)) r[c][i] = 0xff800000u;  // -inf
          }
        }
        const float mx = row_max128(r) * sl2;
        float alpha = 1.f;
        bool rescale = false;
        if (!begun) {
          m_ref = mx;
        } else if (mx > m_ref + kRescaleThreshold) {
          alpha = fast_exp2(m_ref - mx);
          m_ref = mx;
          rescale = true;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // a row with no key seen yet
        const uint64_t sl2_2 = f2_pack(sl2, sl2), negm_2 = f2_pack(-m_use, -m_use);
        uint64_t sum2[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1, e0, e1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1])), sl2_2, negm_2), x0, x1);
            if (HD == 64 && ((i >> 1) & 15) < 6) {
              exp2_pair_poly(x0, x1, e0, e1);
            } else {
              e0 = fast_exp2(x0);
              e1 = fast_exp2(x1);
            }
            sum2[c] = i == 0 ? f2_pack(e0, e1) : f2_add(sum2[c], f2_pack(e0, e1));
            r[c >> 1][(c & 1) * 16 + (i >> 1)] = pack_bf16x2(e0, e1);
          }
        }
        if (begun) {
          // P V of the tile before must be complete before O is rescaled or P overwritten
          if (!(ok = mbar_wait_warp(&pv_done[wg], (n_s - 1) & 1, guard))) break;
          tc_fence_after();
        }
        tmem_st32(tmem + lane_base + colP, r[0]);
        tmem_st32(tmem + lane_base + colP + 32, r[1]);
        if (begun && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + colO + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tmem + lane_base + colO + 32 * c, o);
          }
        }
        float sum_lo, sum_hi;
        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), sum_lo, sum_hi);
        l = l * alpha + (sum_lo + sum_hi);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[wg]);
        begun = true;
        ++n_s;
      }
      if (!ok || !(ok = mbar_wait_warp(&pv_done[wg], (n_s - 1) & 1, guard))) break;
      tc_fence_after();
      const float inv_l = 1.0f / l;
      __nv_bfloat16* dst = args.o + ((static_cast<int64_t>(it.b) * args.T + p) * args.heads + it.head[wg]) * HD;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_base + colO + 32 * c, o);
        tmem_wait_ld();
        if (p < it.n) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 u;
            u.x = pack_bf16x2(__uint_as_float(o[8 * i + 0]) * inv_l, __uint_as_float(o[8 * i + 1]) * inv_l);
            u.y = pack_bf16x2(__uint_as_float(o[8 * i + 2]) * inv_l, __uint_as_float(o[8 * i + 3]) * inv_l);
            u.z = pack_bf16x2(__uint_as_float(o[8 * i + 4]) * inv_l, __uint_as_float(o[8 * i + 5]) * inv_l);
            u.w = pack_bf16x2(__uint_as_float(o[8 * i + 6]) * inv_l, __uint_as_float(o[8 * i + 7]) * inv_l);
            *SAL_CK_ST(d4 + i, 16) = u;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // Every role has finished, so the abort flag is final: let every load this block issued land
  // before the block, and its shared memory, goes away.
  if (warp == 0 && lane == 0 && *abort_flag) {
    for (int i = 0; i < 2; ++i)
      if (loads_q[i] > 0) drain_wait(&q_full[i], (loads_q[i] - 1) & 1);
    for (uint32_t s = 0; s < NS; ++s) {  // the last load of stage s: the largest j < loads with j % NS == s
      if (loads_k > s) drain_wait(&k_full[s], ((loads_k - 1 - s) / NS) & 1);
      if (loads_v > s) drain_wait(&v_full[s], ((loads_v - 1 - s) / NS) & 1);
    }
  }
}

std::mutex g_mu;
int g_sms[64] = {};

template <int HD>
bool prepare_kernel() {
  cudaFuncAttributes fa{};
  return cudaFuncSetAttribute(window_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(Layout<HD>::kSmem)) == cudaSuccess &&
         cudaFuncGetAttributes(&fa, window_kernel<HD>) == cudaSuccess && fa.numRegs * kThreads >= kRegsNeeded &&
         fa.numRegs <= 168;
}

// SMs of the current device once both kernels may run on it (their launch registers must cover
// the split between the warpgroups); 0 if not.
int ready_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_sms[dev]) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !prepare_kernel<128>() ||
        !prepare_kernel<64>())
      return 0;
    g_sms[dev] = sms;
  }
  return g_sms[dev];
}

}  // namespace

sal_status window_attention_launch(const void* q, const void* k, const void* v, int batch, int64_t T, int heads,
                                   int kv_heads, int head_dim, const sal_window& win, const int32_t* lengths, void* o,
                                   cudaStream_t s) {
  const int sms = ready_sms();
  if (!sms) return SAL_ECUDA;
  WindowArgs a{};
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
  a.tiles = (a.T + kTile - 1) / kTile;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(head_dim));
  a.limit_ns = wait_limit_ns();
  a.status = device_status_ptr();
  if (!a.status) return SAL_ECUDA;
  const int planes = batch * heads;
  if (planes * static_cast<int64_t>(a.tiles) <= sms) {
    a.pairing = kSingles;
    a.items = planes * a.tiles;
  } else if ((heads / kv_heads) % 2 == 0) {
    a.pairing = kHeadPairs;
    a.items = planes / 2 * a.tiles;
  } else {
    a.pairing = kTilePairs;
    a.items = planes * ((a.tiles + 1) / 2);
  }
  CUtensorMap tq, tk, tv;
  const uint64_t hd = static_cast<uint64_t>(head_dim), rows = static_cast<uint64_t>(T);
  const uint64_t kvp = static_cast<uint64_t>(batch) * kv_heads;
  if (!make_tmap_3d_bf16(&tq, q, hd, rows, static_cast<uint64_t>(planes), 64, kTile, 1) ||
      !make_tmap_3d_bf16(&tk, k, hd, rows, kvp, 64, kTile, 1) ||
      !make_tmap_3d_bf16(&tv, v, hd, rows, kvp, 64, kTile, 1))
    return SAL_ECUDA;
  ck_declare(o, static_cast<uint64_t>(planes) * rows * hd * 2, true);
  ck_declare(lengths, static_cast<uint64_t>(batch) * 4, false);
  const dim3 grid(static_cast<unsigned>(std::min(sms, a.items)));
  const cudaError_t e =
      head_dim == 128 ? launch_kernel(window_kernel<128>, grid, dim3(kThreads), Layout<128>::kSmem, s, tq, tk, tv, a)
                      : launch_kernel(window_kernel<64>, grid, dim3(kThreads), Layout<64>::kSmem, s, tq, tk, tv, a);
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
