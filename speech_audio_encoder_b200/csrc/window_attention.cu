// Attention with a sliding window and first positions that stay visible (sal_attention_window):
//   o[b, p, h, :] = sum_j a_pj v_j,  a = softmax_j(q_p k_j / sqrt(d)) over the keys j < n_b with
//   j <= p + right and (j >= p - left or j < sinks).
//
// One pass over the visible keys with the running maximum and sum of the softmax, on the tensor
// cores: a tile of 128 query rows takes only the 128-key tiles its rows can see - those of the
// first positions, then those of the window, cut from the first key that is visible - and masks
// single scores only in tiles that a limit cuts. A block holds two query tiles ("slots") that share
// every key tile it loads: two query heads of one key head where heads come in such pairs, else two
// neighbouring tiles of one head (a tile that only one of them sees is skipped by the other). One
// slot alone would read 64 KB of K and V from L2 for every 4 * 128 * 128 * 128 flops, more than L2
// gives all SMs at the tensor core's rate. Where there are no more tiles than SMs each has a block to
// itself (one 30-second clip 7.6 us, as pairs 11.0; 140 tiles 16.9 and 19.4; 200 tiles 27.2 and,
// as pairs, 21.2). Pairs of heads instead of tiles: 271 us for 274 (2 x 8,191 positions, 32 heads on 2).
//
// Windows are short (a minute is six tiles), so starting and ending would cost as much as the
// work: the blocks are persistent, one per SM, and work flows from one item to the next: the
// loads, and the first scores, of the next item go ahead while the rows of this one are stored.
//
// Roles: warp 0 loads keys and queries (TMA); warp 1 issues S = Q K^T for both slots in turn and
// warp 2 O += P V; warp 3 works the items out and loads values; warps 4-7 and 8-11 are the softmax
// of slot 0 and 1, one row per thread. The issuing warps walk in step and elect a lane for each
// instruction: from a branch for one lane every MMA takes 57 clocks to issue, so 15. TMEM: at head dim
// 128 one S (128 columns) that the slots take turns at, O (128) and the weights P (64) of each; at 64
// there is an S for each slot. P is rounded to bf16 for its product, as V is (the row sum is not);
// scores, maxima, sums and O are fp32. O is rescaled only when the maximum grows by more than 8 in
// log2 units (a weight is then at most 256, which fp32 sums and bf16 hold as well as 1).
//
// Measured on one B200, inputs larger than L2: an hour (44,999 positions, 10 heads of 128, 750 back
// and 8 first positions) 259-271 us, 0.65-0.67 PFLOP/s, 40 % of what a large library product reaches
// here; 2 x up to 8,191 positions with 32 heads on 2, 1,023 back, 197-202 us (0.77 PFLOP/s); head dim
// 64, 44,998 x 16, 250 on either side 224-230 us; 16 clips of up to a minute 36 us; 374 positions 7.8 us.
// What bounds it is the softmax's chain: S into registers, maximum, exponentials, P back, with two
// warps per scheduler to hide its latencies; counters of the hour: tensor pipe 41 %, exp2 unit 44 %,
// issue 43 %. A pair of tiles takes about 4,000 clocks, of which the products are 2,080.
// Tried and slower (hour / head dim 64 / grouped, against 274-291 / 223-233 / 212-224 then): P over the
// scores it was made from 428 / 333 / 369; 64-key tiles with an issuer per slot 308 / 263 / 252; sixteen softmax
// warps on half rows each 362 / 267 / 282; one issuing warp 326 / 306 / 281; a copy of the
// loop without masks for whole tiles 312 / 308 / 237 (instruction fetch); 3 in 16 exponentials on the
// FMA pipe 278 / 233 / 218. Items taken in turn with the padded ones among them, 16 clips of up to a
// minute 44 us (36); first positions and the window's first keys in one tile 282 / 242 / 208 (268 / 232 / 201).
#define SAL_CK_FILE 6
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "sal_internal.h"
#include "sal_mma.cuh"

namespace sal {
namespace {

constexpr int kTile = 128;  // query rows of a slot
constexpr int kKeys = 128;  // keys of a tile
constexpr float kRescaleThreshold = 8.0f;  // log2 units: below it the old maximum stays (p <= 256)
constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168, kRegsCtrl = 104, kRegsSoftmax = 200;
static_assert(kRegsCtrl * 128 + kRegsSoftmax * 256 <= kRegsLaunch * kThreads, "the split fits the launch's registers");

template <int HD>
struct Layout {
  static constexpr int kQB = kTile * HD * 2;     // a slot's Q
  static constexpr int kKB = kKeys * HD * 2;     // a tile of K or V
  static constexpr int kBoxes = HD / 64;         // 64-column boxes of a tile
  static constexpr int kBox = 128 * 64 * 2;
  static constexpr int kStagesK = HD == 128 ? 3 : 4, kStagesV = HD == 128 ? 2 : 4;
  static constexpr int kCtrlB = 1024;            // barriers and the work items
  static constexpr size_t kSmem =
      1024 + 2 * static_cast<size_t>(kQB) + (kStagesK + kStagesV) * static_cast<size_t>(kKB) + kCtrlB;
  static constexpr bool kSharedS = HD == 128;    // one score buffer for both slots
  __device__ static uint32_t col_s(int i) { return kSharedS ? 0u : 128u * i; }
  __device__ static uint32_t col_o(int i) { return kSharedS ? 128u + 128u * i : 256u + 64u * i; }
  __device__ static uint32_t col_p(int i) { return 384u + 64u * i; }
};
static_assert(Layout<128>::kSmem <= 227 * 1024 && Layout<64>::kSmem <= 227 * 1024, "shared memory");

constexpr int kItems = 4;  // work items published ahead
enum Pairing { kSingles, kTilePairs, kHeadPairs };

struct WindowArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  const int32_t* lengths;
  int batch, T, heads, kv_heads;
  int left, right, sinks;  // left, right: T for no limit
  int tiles;               // query tiles of a clip
  int pairing, items;
  int wide;                // o is 32-byte aligned
  float scale_log2;
  uint64_t limit_ns;
  unsigned int* status;
  int withhold = -1;       // test hook: key tile of every item from which on no key is loaded
};

// One work item: up to two query tiles and the key tiles they share. Its first tiles hold the
// first positions; the window's tiles start at the first key that any row of the item sees,
// wherever that is (the copies may start at any row), so the fewest tiles cover it. Where the
// first positions reach up to the window the tiles run on from position 0.
struct Item {
  int b, n, kv;         // clip, its length, its (clip, key head) plane
  int head[2], row[2];  // query head and first row of each slot
  int lo[2], hi[2];     // keys [lo, hi) that a slot's window reaches (hi = 0: an empty slot)
  int first, start;     // tiles of first positions, first key of the window's tiles
  int begin[2], last[2];  // the window's tiles [begin, last] that a slot uses, behind those of the first positions
  int count, sinks;     // all tiles; the first positions
  int nth[2];           // items that a slot took part in before this one

  __device__ int base(int x) const { return x < first ? kKeys * x : start + kKeys * (x - first); }
};

// The items of a call in the order of their numbers: those of the longest reach (a causal clip's last
// tiles) first, without those past a clip's end, so that clips of different lengths leave every block
// as many. A whole warp asks for ever higher numbers.
struct Items {
  int rows, per;             // rows of items (one, or a pair, of query tiles each), items of a clip in a row
  int r = 0, before = 0;     // the row it is at, items before it
  int clips, held = 0;       // clips that reach into it (-1: not counted yet); a lane's length where all fit

  __device__ __forceinline__ explicit Items(const WindowArgs& a)
      : rows(a.pairing == kTilePairs ? (a.tiles + 1) / 2 : a.tiles),
        per(a.pairing == kHeadPairs ? a.heads >> 1 : a.heads),
        clips(-1) {
    if (!a.lengths) return;
    int most = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) most = max(most, held = length(a, b0 + (threadIdx.x & 31)));
    most = __reduce_max_sync(0xffffffffu, most);
    r = rows - (most + tile_rows(a) - 1) / tile_rows(a);  // nobody reaches the rows before
  }
  __device__ __forceinline__ static int tile_rows(const WindowArgs& a) { return a.pairing == kTilePairs ? 2 * kTile : kTile; }
  __device__ __forceinline__ static int length(const WindowArgs& a, int b) {
    return b < a.batch ? min(max(*SAL_CK_LD(a.lengths + b, 4), 0), a.T) : 0;
  }
  // the clips b0 + i that reach into row r
  __device__ __forceinline__ uint32_t reach(const WindowArgs& a, int b0) const {
    const int n = a.batch <= 32 ? held : length(a, b0 + (threadIdx.x & 31));
    return __ballot_sync(0xffffffffu, n > (rows - 1 - r) * tile_rows(a));
  }
  // clip, (first) head and (first) query tile of item j; false behind the last
  __device__ __forceinline__ bool find(const WindowArgs& a, int j, int& b, int& h, int& tile) {
    if (!a.lengths) {
      r = j / (a.batch * per);
      before = r * a.batch * per;
    }
    for (;; ++r, before += clips * per, clips = -1) {
      if (r >= rows) return false;
      if (clips < 0) {
        clips = a.lengths ? 0 : a.batch;
        for (int b0 = 0; a.lengths && b0 < a.batch; b0 += 32) clips += __popc(reach(a, b0));
      }
      if (j < before + clips * per) break;
    }
    int rank = (j - before) / per;
    h = (j - before) - rank * per;
    b = rank;
    for (int b0 = 0; a.lengths; b0 += 32) {
      uint32_t in = reach(a, b0);
      const int n = __popc(in);
      if (rank < n) {
        for (; rank > 0; --rank) in &= in - 1;
        b = b0 + __ffs(in) - 1;
        break;
      }
      rank -= n;
    }
    h = a.pairing == kHeadPairs ? 2 * h : h;
    tile = (rows - 1 - r) * (tile_rows(a) / kTile);
    return true;
  }
};

__device__ __forceinline__ Item item_of(const WindowArgs& a, int b, int h, int t0) {
  Item it;
  it.b = b;
  it.n = a.T;
  if (a.lengths) it.n = min(max(*SAL_CK_LD(a.lengths + it.b, 4), 0), a.T);
  it.kv = it.b * a.kv_heads + h / (a.heads / a.kv_heads);
  it.start = 1 << 30;
  int end = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    it.head[i] = h + (a.pairing == kHeadPairs ? i : 0);
    it.row[i] = kTile * (t0 + (a.pairing == kTilePairs ? i : 0));
    it.lo[i] = it.hi[i] = 0;
    if (it.row[i] >= it.n || (i == 1 && a.pairing == kSingles)) continue;
    it.lo[i] = max(0, it.row[i] - a.left);
    it.hi[i] = min(it.n, min(it.row[i] + kTile, it.n) + a.right);
    it.start = min(it.start, it.lo[i]);
    end = max(end, it.hi[i]);
  }
  it.sinks = a.sinks;
  it.first = 0;
  if (a.sinks >= it.start)
    it.start = 0;
  else
    it.first = (a.sinks + kKeys - 1) / kKeys;
  it.count = end > 0 ? it.first + (end - it.start + kKeys - 1) / kKeys : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    it.begin[i] = 0;
    it.last[i] = -1;  // an empty slot uses no tile
    if (it.hi[i] == 0) continue;
    // (where the tiles run on from the first positions, those hold keys for both slots)
    it.begin[i] = it.first + (it.first == 0 && a.sinks > 0 ? 0 : (it.lo[i] - it.start) / kKeys);
    it.last[i] = it.first + (it.hi[i] - 1 - it.start) / kKeys;
  }
  return it;
}

// Maximum of 32 scores held as raw fp32 bits, in two independent chains.
__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
  float m[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t* v = &r[k * 16];
    m[k] = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
    for (int i = 2; i < 16; i += 2) m[k] = max3f(m[k], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
  }
  return fmaxf(m[0], m[1]);
}

// 32 bytes in one store (p 32-byte aligned).
__device__ __forceinline__ void st_global32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Bits [lo, hi) of a 32-bit word (clamped to it).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  lo = max(lo, 0);
  uint32_t r;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(r) : "r"(lo), "r"(max(hi - lo, 0)));
  return r;
}

// Waits (a short time, so without sleep) until a counter in shared memory has reached `need`. A
// whole warp; the bound is checked every 64 polls.
__device__ __forceinline__ bool wait_count(volatile uint32_t* count, uint32_t need, const WaitGuard& g) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1; !__all_sync(0xffffffffu, *count >= need); ++spin) {
    if ((spin & 63) != 0) continue;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(0xffffffffu, *g.abort != 0 || now - t0 > g.limit_ns)) return false;
  }
  return true;
}

// Eight bf16 values as fp32.
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// One row by a warp, straight from memory: row qi of q over the keys [0, lo) and [mid, hi) of the plane
// of keys that begins at row ki, with the maximum and the sum of weights that are known. 32 keys at a
// time, a score to a lane; then every lane adds up its columns.
template <int HD>
__device__ __forceinline__ void sum_row(const WindowArgs& a, int64_t qi, int64_t ki, int lo, int mid, int hi, float m,
                                        float inv_l, __nv_bfloat16* dst) {
  constexpr int kCols = HD / 32;
  const int lane = threadIdx.x & 31, count = lo + max(0, hi - mid);
  float o[kCols] = {};
#pragma unroll 1
  for (int t0 = 0; t0 < count; t0 += 32) {
    const int t = min(t0 + lane, count - 1), j = t < lo ? t : mid + t - lo, n = min(32, count - t0);
    float s = 0.f;
#pragma unroll 8
    for (int d = 0; d < HD / 8; ++d) {
      float x[8], y[8];
      unpack8(*SAL_CK_LD(reinterpret_cast<const uint4*>(a.q + qi * HD) + d, 16), x);
      unpack8(*SAL_CK_LD(reinterpret_cast<const uint4*>(a.k + (ki + j) * HD) + d, 16), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
    }
    const float w = fast_exp2(fmaf(s, a.scale_log2, -m));
#pragma unroll 32
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const int ji = __shfl_sync(0xffffffffu, j, i);
#pragma unroll
      for (int e = 0; e < kCols; e += 2) {
        const uint32_t y =
            *SAL_CK_LD(reinterpret_cast<const uint32_t*>(a.v + (ki + ji) * HD + lane * kCols + e), 4);
        o[e] = fmaf(wi, __uint_as_float(y << 16), o[e]);
        o[e + 1] = fmaf(wi, __uint_as_float(y & 0xffff0000u), o[e + 1]);
      }
    }
    bool lost = true;  // no numbers any more, and so they stay
#pragma unroll
    for (int e = 0; e < kCols; ++e) lost = lost && o[e] != o[e];
    if (__all_sync(0xffffffffu, lost)) break;
  }
#pragma unroll
  for (int e = 0; e < kCols; e += 2)
    *SAL_CK_ST(reinterpret_cast<uint32_t*>(dst + lane * kCols + e), 4) = pack_bf16x2(o[e] * inv_l, o[e + 1] * inv_l);
}

// Whether the lane's row, which sees the keys [lo, hi) and [0, sinks) below hi, does not see one of the
// keys [from, to) that holds a value that is no number. A warp; 32 keys at a time, one to a lane.
template <int HD>
__device__ __forceinline__ bool hides_no_number(const WindowArgs& a, int64_t ki, int from, int to, int sinks, int lo,
                                                int hi) {
  const int lane = threadIdx.x & 31;
  bool hidden = false;
#pragma unroll 1
  for (int j0 = from; j0 < to; j0 += 32) {
    uint32_t bad = 0;
    if (j0 + lane < to) {
#pragma unroll 4
      for (int d = 0; d < HD; d += 8) {
        const uint4 u = *SAL_CK_LD(reinterpret_cast<const uint4*>(a.v + (ki + j0 + lane) * HD + d), 16);
        for (const uint32_t w : {u.x, u.y, u.z, u.w})
          bad |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
      }
    }
    const uint32_t seen = bits_between(lo - j0, hi - j0) | bits_between(0, min(sinks, hi) - j0);
    hidden |= (__ballot_sync(0xffffffffu, bad != 0) & ~seen) != 0;
  }
  return hidden;
}

// The rows in `again` (a lane's row is p) of a warp's 32 that hide a value that is no number among the
// keys of their tiles - those of the window [from, to), and `first` tiles of first positions - summed again.
// An hour, 750 back: one NaN in every head 1.9 to 2.2 ms, only infinities 33 ms (clean 0.25); 8,192
// positions that all see each other and a NaN 0.37 ms, as without (110 if each such row is summed again).
// A function of its own: the same lines inside the loop cost head dim 64 2 % (instruction fetch).
template <int HD>
__device__ __noinline__ void sum_again(const WindowArgs& a, uint32_t again, int b, int head, int kv, int n, int p, int lo,
                                       int hi, int from, int to, int first, float m, float inv_l) {
  const int64_t plane = static_cast<int64_t>(kv) * a.T, rows = (static_cast<int64_t>(b) * a.heads + head) * a.T;
  // keys of the window's tiles in front of what all rows of the warp see, and behind it; and those behind
  // the first positions in their tiles, whether a tile of the window has them too or not
  to = min(n, to);
  const int lo31 = min(to, __shfl_sync(0xffffffffu, lo, 31)), hi0 = __shfl_sync(0xffffffffu, hi, 0);
  bool hidden = false;
#pragma unroll 1
  for (int part = 0; part < (first > 0 ? 3 : 2); ++part)
    hidden |= hides_no_number<HD>(a, plane, part == 0 ? from : part == 1 ? max(max(from, lo31), hi0) : a.sinks,
                                  part == 0 ? lo31 : part == 1 ? to : min(n, (a.sinks + 15) & ~15),
                                  first > 0 ? 0 : a.sinks, part == 2 ? 0 : lo, part == 2 ? 0 : hi);
  again &= __ballot_sync(0xffffffffu, hidden);
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int r = __ffs(again) - 1;
    auto of = [&](auto x) { return __shfl_sync(0xffffffffu, x, r); };
    const int at = of(p), row_lo = of(lo), row_hi = of(hi);
    __syncwarp();  // the row's own stores are behind these
    sum_row<HD>(a, rows + at, plane, min(a.sinks, min(row_lo, row_hi)), row_lo, row_hi, of(m), of(inv_l),
                a.o + ((static_cast<int64_t>(b) * a.T + at) * a.heads + head) * HD);
  }
}

// Where everything is in shared memory.
template <int HD>
struct Shared {
  using L = Layout<HD>;
  uint8_t *q, *k, *v;            // Q0 Q1, K [kStagesK], V [kStagesV]
  uint64_t *q_full, *q_empty;    // [2] Q_i has landed; the item's last S_i has read it
  uint64_t *s_full, *s_free;     // [2] S_i is in its columns; it has been read out of them
  uint64_t *p_full, *pv_done;    // [2] P_i is in place (and O_i rescaled); P_i V is in O_i
  uint64_t* drains;              // [2] wind-down of the issuers
  volatile uint32_t* s_issued;   // [2] S products issued for a slot
  uint64_t *k_full, *k_empty, *v_full, *v_empty;  // per stage: a tile has landed; its last user is done with it
  uint64_t *item_full, *item_empty;               // [kItems] a work item is published; every role is done with it
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  Item* items;                   // [kItems]

  __device__ explicit Shared(uint8_t* base) {
    constexpr int NK = L::kStagesK, NV = L::kStagesV;
    q = base;
    k = base + 2 * L::kQB;
    v = k + NK * L::kKB;
    uint64_t* bars = reinterpret_cast<uint64_t*>(v + NV * L::kKB);
    q_full = bars;
    q_empty = bars + 2;
    s_full = bars + 4;
    s_free = bars + 6;
    p_full = bars + 8;
    pv_done = bars + 10;
    drains = bars + 12;
    s_issued = reinterpret_cast<volatile uint32_t*>(bars + 14);
    k_full = bars + 16;
    k_empty = k_full + NK;
    v_full = k_full + 2 * NK;
    v_empty = v_full + NV;
    item_full = v_full + 2 * NV;
    item_empty = item_full + kItems;
    abort_flag = reinterpret_cast<volatile int*>(item_empty + kItems);
    tmem_slot = reinterpret_cast<uint32_t*>(item_empty + kItems) + 1;
    items = reinterpret_cast<Item*>(reinterpret_cast<uint8_t*>(bars) + 512);
    static_assert((16 + 2 * NK + 2 * NV + 2 * kItems) * 8 + 8 <= 512 && 512 + kItems * sizeof(Item) <= L::kCtrlB,
                  "control block");
  }
};

// What the issuing warps need of an item, in registers: the next product has to be ready to go
// when the buffer it waits for is read.
struct Turn {
  int count, first, start, sinks, begin0, begin1, last0, last1, hi0, hi1;
  __device__ void load(const Item& it) {
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    count = same(it.count);
    first = same(it.first);
    start = same(it.start);
    sinks = same(it.sinks);
    begin0 = same(it.begin[0]);
    begin1 = same(it.begin[1]);
    last0 = same(it.last[0]);
    last1 = same(it.last[1]);
    hi0 = same(it.hi[0]);
    hi1 = same(it.hi[1]);
  }
  // tiles of slot i, and the r-th of them
  __device__ int tiles(int i) const { return i ? (last1 < 0 ? 0 : first + last1 + 1 - begin1) : (last0 < 0 ? 0 : first + last0 + 1 - begin0); }
  __device__ int tile(int i, int r) const { return r < first ? r : (i ? begin1 : begin0) + r - first; }
  // whether slot i is the last to take tile x: where both do, slot 1 unless it comes to it a turn earlier
  __device__ bool frees(int i, int x, int lag) const {
    const bool other = i ? x <= last0 && (x < first || x >= begin0) : x <= last1 && (x < first || x >= begin1);
    return !other || i == (x < first || begin1 == begin0 + lag ? 1 : 0);
  }
  __device__ int base(int x) const { return x < first ? kKeys * x : start + kKeys * (x - first); }
  // keys of tile x that slot i multiplies with: a multiple of 16, the rest of the tile is not used
  __device__ int cols(int i, int x) const {
    return min(kKeys, ((x < first ? sinks : i ? hi1 : hi0) - base(x) + 15) & ~15);
  }
};

// S = Q K^T for slot 0 and slot 1 in turn, each for the next of its own tiles, as soon as the
// buffer has been read. (In the order of the tiles, a tile that only one slot takes would give
// that slot two turns in a row, and the second would hold the buffer until its softmax is done
// with the first.) A whole warp walks in step; one of its lanes issues.
template <int HD>
__device__ __forceinline__ bool issue_scores(const Shared<HD>& sm, const WaitGuard& guard, uint32_t tmem) {
  using L = Layout<HD>;
  constexpr uint32_t IDESC_S = idesc_bf16(128, 0, false, false);  // + columns / 8 << 17
  const uint32_t one = elect_one();
  const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(sm.q)), k_desc = sdesc_kmajor_sw128(smem_u32(sm.k));
  constexpr uint32_t NK = L::kStagesK;
  uint32_t tile0 = 0, landed = 0;                    // tiles of the items before, tiles known to have landed
  uint32_t n0 = 0, n1 = 0, q0 = 0, q1 = 0;           // S products and items of each slot so far
  Turn t;
  for (int k = 0;; ++k) {
    if (!mbar_sleep_warp(&sm.item_full[k % kItems], (k / kItems) & 1, guard)) return false;
    t.load(sm.items[k % kItems]);
    __syncwarp();
    if (one) mbar_arrive(&sm.item_empty[k % kItems]);
    if (t.count == 0) return true;
    const int tiles0 = t.tiles(0), tiles1 = t.tiles(1);
    const int lag = L::kSharedS ? 0 : t.begin1 - t.begin0;
    for (int turn = 0; turn < max(tiles0, tiles1 + lag); ++turn) {
#pragma unroll 1
      for (int i = turn < tiles0 ? 0 : 1; i < (turn >= lag && turn - lag < tiles1 ? 2 : 1); ++i) {
        const int r = i ? turn - lag : turn;
        const int x = t.tile(i, r);
        const uint32_t stage = (tile0 + x) % NK, par = (tile0 + x) / NK & 1;
        const uint32_t idesc = IDESC_S | (static_cast<uint32_t>(t.cols(i, x)) >> 3 << 17), d = tmem + L::col_s(i);
        const uint64_t qd = q_desc + i * (L::kQB / 16), kd = k_desc + stage * (L::kKB / 16);
        const uint32_t mine = i ? n1 : n0, before = L::kSharedS ? n0 + n1 : mine;
        const bool frees = t.frees(i, x, lag), ends = r + 1 == (i ? tiles1 : tiles0);
        if (tile0 + x >= landed) {  // (once a tile: even a wait that is over takes about 100 clocks)
          if (!mbar_sleep_warp(&sm.k_full[stage], par, guard)) return false;
          landed = tile0 + x + 1;
        }
        if (r == 0 && !mbar_sleep_warp(&sm.q_full[i], (i ? q1 : q0) & 1, guard)) return false;
        // the scores before it have been read out of the buffer
        if (before > 0 && !mbar_sleep_warp(&sm.s_free[L::kSharedS ? 0 : i], (before - 1) & 1, guard)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          umma_ss_one(one, d, qd + (kk >> 2) * (L::kBox / 16) + (kk & 3) * 2,
                      kd + (kk >> 2) * (L::kBox / 16) + (kk & 3) * 2, idesc, kk > 0);
        umma_commit_one(one, &sm.s_full[i]);
        if (one) sm.s_issued[i] = mine + 1;
        if (frees) umma_commit_one(one, &sm.k_empty[stage]);
        if (ends) umma_commit_one(one, &sm.q_empty[i]);
        if (i)
          ++n1;
        else
          ++n0;
      }
    }
    q0 += tiles0 > 0;
    q1 += tiles1 > 0;
    tile0 += t.count;
  }
}

// O += P V in the same order, by a warp of its own (its lanes clear the rows of V past a clip's
// end). The tensor core runs products in the order they are issued: a slot's next S, which its
// softmax waits for, goes ahead of its P V.
template <int HD>
__device__ __forceinline__ bool issue_outputs(const WindowArgs& args, const Shared<HD>& sm, const WaitGuard& guard,
                                              uint32_t tmem) {
  using L = Layout<HD>;
  constexpr uint32_t IDESC_O = idesc_bf16(128, HD, false, true);
  const uint32_t lane = threadIdx.x & 31, one = elect_one();
  const uint64_t v_desc = sdesc_mnmajor_sw128(smem_u32(sm.v), L::kBox);
  constexpr uint32_t NV = L::kStagesV;
  uint32_t tile0 = 0, landed = 0, n0 = 0, n1 = 0;  // tiles of the items before and landed; P V products of each slot
  Turn t;
  for (int k = 0;; ++k) {
    if (!mbar_sleep_warp(&sm.item_full[k % kItems], (k / kItems) & 1, guard)) return false;
    t.load(sm.items[k % kItems]);
    const int n = __shfl_sync(0xffffffffu, sm.items[k % kItems].n, 0);
    __syncwarp();
    if (one) mbar_arrive(&sm.item_empty[k % kItems]);
    if (t.count == 0) return true;
    const int tiles0 = t.tiles(0), tiles1 = t.tiles(1);
    const int lag = L::kSharedS ? 0 : t.begin1 - t.begin0;
    for (int turn = 0; turn < max(tiles0, tiles1 + lag); ++turn) {
#pragma unroll 1
      for (int i = turn < tiles0 ? 0 : 1; i < (turn >= lag && turn - lag < tiles1 ? 2 : 1); ++i) {
        const int r = i ? turn - lag : turn;
        const int x = t.tile(i, r), cols = t.cols(i, x), clear = n < args.T ? n - t.base(x) : kKeys;
        const uint32_t stage = (tile0 + x) % NV, par = (tile0 + x) / NV & 1;
        const uint64_t vd = v_desc + stage * (L::kKB / 16);
        const uint32_t mine = i ? n1 : n0, d = tmem + L::col_o(i), pa = tmem + L::col_p(i);
        const bool frees = t.frees(i, x, lag), ends = r + 1 == (i ? tiles1 : tiles0);
        if (tile0 + x >= landed) {
          if (!mbar_sleep_warp(&sm.v_full[stage], par, guard)) return false;
          landed = tile0 + x + 1;
        }
        if (clear < cols) {
          // rows past the clip's length hold anything (NaN times a weight of zero is NaN): zeros. (The
          // other slot may write the same zeros while this one's product reads them.)
          for (int j = clear + (lane >> 3); j < cols; j += 4)
            for (int b = 0; b < L::kBoxes; ++b)
              *reinterpret_cast<uint4*>(sm.v + stage * L::kKB + b * L::kBox + j * 128 + (lane & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!mbar_sleep_warp(&sm.p_full[i], mine & 1, guard)) return false;
        if (!ends && !wait_count(&sm.s_issued[i], mine + 2, guard)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          if (kk * 16 < cols) umma_ts_one(one, d, pa + kk * 8, vd + kk * (2048 / 16), IDESC_O, (r > 0 || kk > 0));
        umma_commit_one(one, &sm.pv_done[i]);
        if (frees) umma_commit_one(one, &sm.v_empty[stage]);
        if (i)
          ++n1;
        else
          ++n0;
      }
    }
    tile0 += t.count;
  }
}

// Behind an issuing warp whose wait gave up, or whose block is winding down: its products still in
// flight complete before the block's tensor memory goes.
__device__ __forceinline__ void drain_products(uint64_t* bar, bool ok, const WaitGuard& guard) {
  if (!ok) give_up(guard);
  if (*guard.abort) {
    const uint32_t one = elect_one();
    umma_commit_one(one, bar);
    if (one) drain_wait(bar, 0);
  }
  __syncwarp();
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WindowArgs args) {
  using L = Layout<HD>;
  constexpr int NK = L::kStagesK, NV = L::kStagesV;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Shared<HD> sm(smem);
  uint64_t *const q_full = sm.q_full, *const q_empty = sm.q_empty, *const s_full = sm.s_full, *const s_free = sm.s_free;
  uint64_t *const p_full = sm.p_full, *const pv_done = sm.pv_done, *const k_full = sm.k_full, *const k_empty = sm.k_empty;
  uint64_t *const v_full = sm.v_full, *const v_empty = sm.v_empty, *const item_full = sm.item_full;
  uint64_t* const item_empty = sm.item_empty;
  uint8_t *const sQ = sm.q, *const sK = sm.k, *const sV = sm.v;
  volatile int* const abort_flag = sm.abort_flag;
  uint32_t* const tmem_slot = sm.tmem_slot;
  Item* const items = sm.items;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);  // one arrival per softmax warp of the slot
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&sm.drains[i], 1);
      sm.s_issued[i] = 0;
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 11);  // loader, two issuers, eight softmax warps
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const WaitGuard guard{abort_flag, args.limit_ns, args.status};
  // the loaders' records of what they have loaded, for the wind-down
  uint32_t loads_q[2] = {0, 0}, loads_k = 0, loads_v = 0;
  bool ok = true;
  // Waits for the k-th work item of this block; done_with lets its place be reused.
  auto item_ready = [&](int k) { return mbar_sleep(&item_full[k % kItems], (k / kItems) & 1, guard); };
  auto done_with = [&](int k) { mbar_arrive(&item_empty[k % kItems]); };

  // Each role runs inside the branch that set its register limit.
  if (warp < 4) {
    setmaxnreg_dec<kRegsCtrl>();
  if (warp == 0) {
    pdl_wait();  // (each role waits for the kernel before where it first touches memory)
    if (lane == 0) {
      // keys, and behind an item's first tile its queries, as soon as the last S before has read its slot's
      bool go = true;
      for (int k = 0; ok && go; ++k) {
        if (!(ok = item_ready(k))) break;
        const Item& it = items[k % kItems];
        if (it.count == 0) break;
        for (int x = 0; ok && x < it.count; ++x) {
          if (!(go = x != args.withhold)) break;
          const uint32_t s = loads_k % NK;
          if (!(ok = mbar_sleep(&k_empty[s], ((loads_k / NK) & 1) ^ 1, guard))) break;
          mbar_arrive_expect_tx(&k_full[s], L::kKB);
          for (int b = 0; b < L::kBoxes; ++b)
            tma_load_3d(sK + s * L::kKB + b * L::kBox, &tmK, &k_full[s], 64 * b, it.base(x), it.kv);
          ++loads_k;
          for (int i = 0; x == 0 && ok && i < 2; ++i) {
            if (it.hi[i] == 0) continue;
            if (!(ok = mbar_sleep(&q_empty[i], (it.nth[i] & 1) ^ 1, guard))) break;
            mbar_arrive_expect_tx(&q_full[i], L::kQB);
            for (int b = 0; b < L::kBoxes; ++b)
              tma_load_3d(sQ + i * L::kQB + b * L::kBox, &tmQ, &q_full[i], 64 * b, it.row[i],
                          it.b * args.heads + it.head[i]);
            loads_q[i] = it.nth[i] + 1;
          }
        }
        done_with(k);
      }
    }
  } else if (warp == 1) {
    drain_products(&sm.drains[0], issue_scores<HD>(sm, guard, tmem), guard);
  } else if (warp == 2) {
    drain_products(&sm.drains[1], issue_outputs<HD>(args, sm, guard, tmem), guard);
  } else if (warp == 3) {
    if (args.lengths) pdl_wait();
    // works the items out one ahead of the other roles (an item of no tiles is the end), and loads the
    // values: a thread of its own, so that a key tile never waits for a value tile's place
    Items list(args);
    int nth[2] = {0, 0};
    Item now, next;
    for (int k = -1; __shfl_sync(0xffffffffu, ok, 0); ++k) {
      int b, h, t0;
      // to and fro over the blocks, so that no block gets the longest of every round
      const int round = k + 1, at_block = round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
      const bool more = list.find(args, round * static_cast<int>(gridDim.x) + at_block, b, h, t0);
      if (lane == 0) {
        next.count = 0;
        if (more) next = item_of(args, b, h, t0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          next.nth[i] = nth[i];
          nth[i] += next.count > 0 && next.hi[i] > 0;
        }
        const int at = (k + 1) % kItems;
        if ((ok = mbar_sleep(&item_empty[at], (((k + 1) / kItems) & 1) ^ 1, guard))) {
          items[at] = next;
          mbar_arrive(&item_full[at]);
        }
        if (k < 0) pdl_wait();
        if (k >= 0) {
          for (int x = 0; ok && x < now.count; ++x) {
            const uint32_t s = loads_v % NV;
            if (!(ok = mbar_sleep(&v_empty[s], ((loads_v / NV) & 1) ^ 1, guard))) break;
            mbar_arrive_expect_tx(&v_full[s], L::kKB);
            for (int b = 0; b < L::kBoxes; ++b)
              tma_load_3d(sV + s * L::kKB + b * L::kBox, &tmV, &v_full[s], 64 * b, now.base(x), now.kv);
            ++loads_v;
          }
        }
        now = next;
      }
      if (!more) break;
    }
  }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    pdl_wait();
    const int slot = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t colS = tmem + lane_base + L::col_s(slot), colP = tmem + lane_base + L::col_p(slot);
    const uint32_t colO = tmem + lane_base + L::col_o(slot);
    const int row = quarter * 32 + lane;
    const float sl2 = args.scale_log2;
    uint32_t n_s = 0;  // score tiles of this slot so far
    for (int k = 0; ok; ++k) {
      if (!(ok = mbar_sleep_warp(&item_full[k % kItems], (k / kItems) & 1, guard))) break;
      const Item& it = items[k % kItems];
      if (it.count == 0) break;
      const int p = it.row[slot] + row;
      const int key_lo = max(0, p - args.left), key_hi = min(it.n, p + args.right + 1);
      float m_ref = -INFINITY, l = 0.f;
      bool begun = false;
      const int first = it.first, begin = it.begin[slot], last = it.last[slot], start = it.start;
      for (int x = first > 0 ? 0 : begin; x <= last; x = x + 1 == first ? begin : x + 1) {
        if (!(ok = mbar_sleep_warp(&s_full[slot], n_s & 1, guard))) break;
        tc_fence_after();
        uint32_t r[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(colS + 32 * c, r[c]);
        const int base = x < first ? kKeys * x : start + kKeys * (x - first);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[L::kSharedS ? 0 : slot]);  // back to the tensor core
        // P V of the tile before must be complete before O is rescaled or P overwritten (asked for here,
        // needed below)
        const bool pv_ok = n_s == 0 || mbar_test(&pv_done[slot], (n_s - 1) & 1);
        // halves of the tile that some row of the warp sees (the others cost nothing below)
        uint32_t live = 3u;
        if (__any_sync(0xffffffffu, x < first || base < key_lo || base + kKeys > key_hi)) {
          // a tile of first positions ends at the last of them; where the tiles run on from position 0
          // the first positions add to the window's
          const bool early = x < first;
          const int extra = early || first > 0 ? 0 : args.sinks;
          live = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = base + 32 * c;
            const uint32_t seen = early ? bits_between(0, args.sinks - at)
                                        : bits_between(key_lo - at, key_hi - at) | bits_between(0, min(extra, key_hi) - at);
            if (__any_sync(0xffffffffu, seen != 0)) live |= 1u << (c >> 1);
            if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((seen >> i) & 1u)) r[c][i] = 0xff800000u;  // -inf
            }
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((live >> h) & 1u) mx = fmaxf(mx, fmaxf(max32(r[2 * h]), max32(r[2 * h + 1])));
        mx *= sl2;
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
        uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if ((live >> h) & 1u) {
#pragma unroll
            for (int c = 2 * h; c < 2 * h + 2; ++c) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1])), sl2_2, negm_2), x0,
                          x1);
                const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                sum2[c] = i == 0 ? f2_pack(e0, e1) : f2_add(sum2[c], f2_pack(e0, e1));
                r[h][(c & 1) * 16 + (i >> 1)] = pack_bf16x2(e0, e1);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[h][i] = 0;
          }
        }
        if (!__all_sync(0xffffffffu, pv_ok) && !(ok = mbar_sleep_warp(&pv_done[slot], (n_s - 1) & 1, guard))) break;
        tc_fence_after();
        tmem_st32(colP, r[0]);
        tmem_st32(colP + 32, r[1]);
        if (begun && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(colO + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(colO + 32 * c, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[slot]);
        float sum_lo, sum_hi;
        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), sum_lo, sum_hi);
        l = l * alpha + (sum_lo + sum_hi);
        begun = true;
        ++n_s;
      }
      if (!ok) break;
      const int n = it.n;
      const bool stored = p < n;
      const int head = it.head[slot], b = it.b, kv = it.kv;
      __nv_bfloat16* dst = args.o + ((static_cast<int64_t>(b) * args.T + p) * args.heads + head) * HD;
      __syncwarp();
      if (lane == 0) done_with(k);
      if (!begun) continue;  // an empty slot
      if (!(ok = mbar_sleep_warp(&pv_done[slot], (n_s - 1) & 1, guard))) break;
      tc_fence_after();
      const float inv_l = 1.0f / l;
      uint64_t zeros[4] = {0, 0, 0, 0};  // zero times every value of the row
#pragma unroll 1
      for (int c = 0; c < HD / 64; ++c) {
        uint32_t u[2][32];
        tmem_ld32(colO + 64 * c, u[0]);
        tmem_ld32(colO + 64 * c + 32, u[1]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          uint64_t& z = zeros[(i >> 1) & 3];
          z = f2_fma(f2_pack(__uint_as_float(u[i >> 5][i & 31]), __uint_as_float(u[i >> 5][(i & 31) + 1])), 0, z);
        }
        if (stored) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            u[0][i] = pack_bf16x2(__uint_as_float(u[i >> 4][2 * (i & 15)]) * inv_l,
                                  __uint_as_float(u[i >> 4][2 * (i & 15) + 1]) * inv_l);
          if (args.wide) {  // a whole 32-byte sector at a time
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global32(SAL_CK_ST(dst + 64 * c + 16 * i, 32), &u[0][8 * i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *SAL_CK_ST(reinterpret_cast<uint4*>(dst + 64 * c) + i, 16) =
                  make_uint4(u[0][4 * i], u[0][4 * i + 1], u[0][4 * i + 2], u[0][4 * i + 3]);
          }
        }
      }
      float zero_lo, zero_hi;
      f2_unpack(f2_add(f2_add(zeros[0], zeros[1]), f2_add(zeros[2], zeros[3])), zero_lo, zero_hi);
      // A value that is no number, at a key of these tiles that the row does not see, has met a weight of
      // zero: such a row is summed again over what it does see. (One that only sees such values, or whose
      // weights are no numbers, is as it should be.)
      const uint32_t again = __ballot_sync(0xffffffffu, stored && l == l && !(zero_lo + zero_hi == 0.f));
      if (again)
        sum_again<HD>(args, again, b, head, kv, n, p, key_lo, key_hi, start + kKeys * (begin - first),
                      start + kKeys * (last - first + 1), first, m_ref == -INFINITY ? 0.f : m_ref, inv_l);
      // (O is overwritten by the next item's first product, which waits for this slot's next P)
    }
  }

  if (!ok) give_up(guard);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // Every role has finished, so the abort flag is final: let every load this block issued land
  // before the block, and its shared memory, goes away.
  if ((warp == 0 || warp == 3) && lane == 0 && *abort_flag) {
    for (int i = 0; i < 2; ++i)
      if (loads_q[i] > 0) drain_wait(&q_full[i], (loads_q[i] - 1) & 1);
    // the last load of stage s: the largest j < loads with j % stages == s
    for (uint32_t s = 0; s < NK; ++s)
      if (loads_k > s) drain_wait(&k_full[s], ((loads_k - 1 - s) / NK) & 1);
    for (uint32_t s = 0; s < NV; ++s)
      if (loads_v > s) drain_wait(&v_full[s], ((loads_v - 1 - s) / NV) & 1);
  }
}

std::mutex g_mu;
int g_sms[64] = {};

template <int HD>
bool prepare_kernel() {
  cudaFuncAttributes fa{};
  return cudaFuncSetAttribute(window_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(Layout<HD>::kSmem)) == cudaSuccess &&
         cudaFuncGetAttributes(&fa, window_kernel<HD>) == cudaSuccess && fa.numRegs == kRegsLaunch;
}

// SMs of the current device once both kernels may run on it; 0 if not.
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
                                   cudaStream_t s, int withhold) {
  const int sms = ready_sms();
  if (!sms) return SAL_ECUDA;
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
  a.tiles = (a.T + kTile - 1) / kTile;
  a.wide = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(head_dim));
  a.limit_ns = wait_limit_ns();
  a.withhold = withhold;
  a.status = device_status_ptr();
  if (!a.status) return SAL_ECUDA;
  const int planes = batch * heads;
  if (planes * static_cast<int64_t>(a.tiles) <= sms) {  // (times of both sides of these rules: above)
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
      !make_tmap_3d_bf16(&tk, k, hd, rows, kvp, 64, kKeys, 1) ||
      !make_tmap_3d_bf16(&tv, v, hd, rows, kvp, 64, kKeys, 1))
    return SAL_ECUDA;
  ck_declare(q, static_cast<uint64_t>(planes) * rows * hd * 2, false);
  ck_declare(k, kvp * rows * hd * 2, false);
  ck_declare(v, kvp * rows * hd * 2, false);
  ck_declare(o, static_cast<uint64_t>(planes) * rows * hd * 2, true);
  ck_declare(lengths, static_cast<uint64_t>(batch) * 4, false);
  const dim3 grid(static_cast<unsigned>(std::min(sms, a.items)));
  const cudaError_t e =
      head_dim == 128 ? launch_kernel(window_kernel<128>, grid, dim3(kThreads), Layout<128>::kSmem, s, tq, tk, tv, a)
                      : launch_kernel(window_kernel<64>, grid, dim3(kThreads), Layout<64>::kSmem, s, tq, tk, tv, a);
  return e == cudaSuccess ? SAL_OK : SAL_ECUDA;
}

}  // namespace sal

namespace {
sal_status attention_window(const void* q, const void* k, const void* v, int batch, int64_t T, int heads, int kv_heads,
                            int head_dim, const sal_window* window, const int32_t* lengths, void* o, void* stream,
                            int withhold) {
  using namespace sal;
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
                                 static_cast<cudaStream_t>(stream), withhold);
}
}  // namespace

extern "C" sal_status sal_attention_window(const void* q, const void* k, const void* v, int batch, int64_t T,
                                           int heads, int kv_heads, int head_dim, const sal_window* window,
                                           const int32_t* lengths, void* o, void* stream) {
  const sal::NvtxRange nvtx_("sal_attention_window");
  return attention_window(q, k, v, batch, T, heads, kv_heads, head_dim, window, lengths, o, stream, -1);
}

// Test hook: no key tile of an item from `tile` on is loaded, so that bounded waits give up (see sal.h).
extern "C" sal_status sal_attention_window_withhold(const void* q, const void* k, const void* v, int batch, int64_t T,
                                                    int heads, int head_dim, const sal_window* window, int tile,
                                                    void* o, void* stream) {
  const sal::NvtxRange nvtx_("sal_attention_window_withhold");
  if (tile < 0) return SAL_EINVAL;
  return attention_window(q, k, v, batch, T, heads, heads, head_dim, window, nullptr, o, stream, tile);
}
