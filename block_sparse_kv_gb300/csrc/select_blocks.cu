// Blocks of a paged cache chosen for each query by a bound of its logits, and the bounds they are
// chosen by. A block is a page.
//
// Bounds: per page and kv head the least and the greatest value of each key channel over the page's
// tokens, lo_d and hi_d. They are values of the cache, so nothing is rounded.
//
// Score. For a query head q and any key k of the block, q.k <= sum_d max(q_d lo_d, q_d hi_d). The
// blocks of a kv head serve its whole group, so a block's score is that bound summed over the heads of
// the group, and since lo_d <= hi_d
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d hi_d P_d + lo_d N_d,
//   P_d = sum_h max(q_hd, 0),  N_d = sum_h min(q_hd, 0):
// one product of 2 D values per block however many heads there are. That is far below what the ALUs
// can do per byte, so scoring is bound by reading the bounds once. Where a bound is infinite the folded form has
// products of it with coefficients of zero, NaN, that the sum over heads does not have; rows with such values, which
// their error bound shows, are scored again by the CTA that selects from them.
//
// Selection. The first `sink` and the last `recent` blocks that a query sees stay, and of the others the k of
// highest score, as 64-bit arithmetic would choose them (the lowest index among equals). Scores are summed in
// fp32 with an error of at most E = (group + 10) 2^-24 sum_d max_j |hi_jd| P_d + max_j |lo_jd| |N_d|: coefficients
// are sums of up to `group` terms, a lane's eight products two chains of four, six more additions join them.
// With s_k the k-th largest fp32 score, blocks above s_k + 2 E are chosen and those below s_k - 2 E are
// not, whatever the rounding; only the blocks between are scored again, in fp64 (a few us for the few rows that need
// it). Rows where nothing lies between but as many blocks as are still wanted (nearly all) need no second look.
//
// Two launches, the second ready to go when the first ends: scoring keeps the memory busy only while all SMs score.
// With the selection by the CTA that finished a row's last part the operator took 56 us for 64 requests of 2048 to
// 16384 tokens and 31 for one of 131072 (8 kv heads, blocks of 16), in two launches 43 and 19.
#include <algorithm>
#include <type_traits>

#include "cache_common.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------------------
// bounds of touched pages
// ---------------------------------------------------------------------------------------

constexpr int kBoundsThreads = 256;
constexpr int kBoundsCtas = 3;   // per SM
constexpr int kBoundsRows = 32;  // most token rows that a warp looks at
constexpr int kBoundsStages = 2;
constexpr int kBoundsAhead = 8;  // 16-byte copies of a lane at a time

struct BoundsParams {
  const uint8_t* keys;
  int64_t k_s0, k_s2, k_s3;  // bytes: page, kv head, slot
  uint8_t* bounds;
  int64_t b_s0, b_s1;        // bytes: page, kv head
  const int32_t *batch_indices, *positions, *kv_indptr, *kv_indices, *kv_last_page_len;
  int64_t nnz;
  int heads, batch, num_pages, rows;
  int units;  // groups of rows times kv heads
  FastDiv page_size, by_head;
  StatusArgs st;
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f807f80u, kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // the larger absolute values, with some sign; a number rather than NaN
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float2 values(uint32_t a) {
    return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
  // 0xffff in the halves of numbers below infinity, and of all but infinity; `a` without its signs
  static __device__ __forceinline__ uint32_t finite(uint32_t a) { return __hlt2_mask(half2_of(a), half2_of(kInf)); }
  static __device__ __forceinline__ uint32_t not_infinite(uint32_t a) { return __hneu2_mask(half2_of(a), half2_of(kInf)); }
  static __device__ __forceinline__ __nv_bfloat162 half2_of(uint32_t a) { return *reinterpret_cast<__nv_bfloat162*>(&a); }
};
template <>
struct Pair<__half> {
  static constexpr uint32_t kInf = 0x7c007c00u, kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float2 values(uint32_t a) {
    return __half22float2(*reinterpret_cast<const __half2*>(&a));
  }
  static __device__ __forceinline__ uint32_t finite(uint32_t a) { return __hlt2_mask(half2_of(a), half2_of(kInf)); }
  static __device__ __forceinline__ uint32_t not_infinite(uint32_t a) { return __hneu2_mask(half2_of(a), half2_of(kInf)); }
  static __device__ __forceinline__ __half2 half2_of(uint32_t a) { return *reinterpret_cast<__half2*>(&a); }
};

// What the copying side tells the computing side about a stage.
struct BoundsInfo {
  int page, head;
  int left;   // slots of the page from the stage's first on
  int flags;  // 1: first round of the page, 2: last
};

// A warp looks at `rows` token rows for one kv head at a time. A page is done for each row that is its first
// among consecutive rows: in whatever order the rows are, the lowest position of a page is one of those, and a
// page that is done twice gets the same bytes. Bound by reading the keys: a row is D / 8 lanes of 16 bytes, and
// the rows of up to 16 slots are copied while those before them are compared (32000 tokens of 8 heads in pages of 16:
// 16.1 us, 4.6 TB/s of keys and bounds; by CTAs of 32 rows with loads in registers 20.4).
template <typename T, int D>
__global__ void __launch_bounds__(kBoundsThreads, kBoundsCtas) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kLanes = D / 8, kSlots = 32 / kLanes, kRound = kSlots * kBoundsAhead, kWarps = kBoundsThreads / 32;
  extern __shared__ uint4 ring[];
  __shared__ BoundsInfo infos[kWarps][kBoundsStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % kLanes, slot0 = lane / kLanes;
  uint4* mine = ring + warp * (kBoundsStages * kBoundsAhead * 32) + lane;
  const int step = gridDim.x * kWarps;
  int unit = blockIdx.x * kWarps + warp - step;
  // the unit's pages that are to be done: lane i's row has page `page` with `fill` tokens
  uint32_t todo = 0;
  int page = -1, fill = 0, head = 0;
  // the page that is being copied: slots [slot, n)
  int pg = 0, slot = 0, n = 0;
  auto look = [&]() {
    const int64_t i = int64_t(p.by_head.divmod(unit, head)) * p.rows + lane;
    page = -1;
    if (lane < p.rows && i < p.nnz) {
      const int b = __ldg(p.batch_indices + i), pos = __ldg(p.positions + i);
      const int b0 = i > 0 ? __ldg(p.batch_indices + i - 1) : -1, pos0 = i > 0 ? __ldg(p.positions + i - 1) : 0;
      int in_page = 0;
      const int j = pos >= 0 ? p.page_size.divmod(pos, in_page) : 0;
      const bool before = b0 == b && pos0 == pos - 1;
      if (b >= 0 && (in_page == 0 || !before || pos < 0)) {
        bool bad = b >= p.batch || pos < 0;
        if (!bad) {
          const int start = __ldg(p.kv_indptr + b), count = __ldg(p.kv_indptr + b + 1) - start;
          bad = j >= count;
          if (!bad) {
            page = __ldg(p.kv_indices + start + j);
            fill = j == count - 1 ? __ldg(p.kv_last_page_len + b) : int(p.page_size.d);
            bad = page < 0 || page >= p.num_pages || fill < 1 || fill > int(p.page_size.d);
          }
        }
        if (bad) {
          record_error(p.st, BSKV_ERR_DEVICE_INDEX);
          page = -1;
        }
      }
    }
    todo = __ballot_sync(0xffffffffu, page >= 0);
  };
  int issued = 0;
  auto issue = [&]() {
    while (slot >= n && (todo || unit + step < p.units)) {
      if (!todo) {
        unit += step;
        look();
        continue;
      }
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      pg = __shfl_sync(0xffffffffu, page, src);
      n = __shfl_sync(0xffffffffu, fill, src);
      slot = 0;
    }
    if (slot < n) {
      const int stage = issued % kBoundsStages;
      const uint8_t* from = p.keys + pg * p.k_s0 + head * p.k_s2 + (slot + slot0) * p.k_s3 + 16 * sub;
#pragma unroll
      for (int u = 0; u < kBoundsAhead; ++u) {
        if (slot + slot0 + u * kSlots < n) cp_async_16(mine + (stage * kBoundsAhead + u) * 32, from);
        from += kSlots * p.k_s3;
      }
      if (lane == 0) infos[warp][stage] = BoundsInfo{pg, head, n - slot, (slot == 0 ? 1 : 0) | (slot + kRound >= n ? 2 : 0)};
      slot += kRound;
      ++issued;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kBoundsStages - 1; ++i) issue();
  uint32_t lo[4], hi[4];
  for (int consumed = 0; consumed < issued; ++consumed) {
    __syncwarp();  // the stage that is filled next has been read, and its round is described
    const int stage = consumed % kBoundsStages;
    const BoundsInfo info = infos[warp][stage];
    issue();
    cp_async_wait<kBoundsStages - 1>();
    if (info.flags & 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = Pair<T>::kInf;
        hi[c] = Pair<T>::kNegInf;
      }
    }
#pragma unroll
    for (int u = 0; u < kBoundsAhead; ++u) {
      if (slot0 + u * kSlots >= info.left) continue;
      const uint4 x = mine[(stage * kBoundsAhead + u) * 32];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = Pair<T>::low(lo[c], w[c]);
        hi[c] = Pair<T>::high(hi[c], w[c]);
      }
    }
    if (!(info.flags & 2)) continue;
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = Pair<T>::low(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], o));
        hi[c] = Pair<T>::high(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], o));
      }
    }
    // lo, then hi: 2 kLanes lanes write
    if (lane < 2 * kLanes)
      *reinterpret_cast<uint4*>(p.bounds + info.page * p.b_s0 + info.head * p.b_s1 + 16 * lane) =
          lane >= kLanes ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---------------------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------------------

constexpr int kScoreThreads = 256;
constexpr int kScoreCtas = 2;  // per SM
constexpr int kScoreStages = 3;
constexpr int kAhead = 8;      // 16-byte loads of a lane at a time
constexpr int kKept = 1024;    // queries whose rows fit in shared memory beside the rings
constexpr int kBins = 256;
constexpr int kFew = 64;     // keys that are ranked one against the other

struct SelectParams {
  const void* q;
  int64_t q_s0, q_s1;
  const uint8_t* bounds;
  int64_t b_s0, b_s1;  // bytes: page, kv head
  const int32_t *batch_indices, *positions, *kv_indptr, *kv_indices;
  int32_t* blocks;
  float* scores;               // [rows][stride]; then the upper halves of fp64 scores' keys
  unsigned* most;              // [rows]: bounds of the sums of absolute products, zero between runs
  int group, batch, num_pages, max_blocks, stride, top_k, sink, recent;
  int queries;
  int set_heads, sets, head_groups;  // scoring: warps (kv heads) of a set, sets of a CTA, sets' worth of heads
  FastDiv page_size, heads;
  float error;                 // E over that bound
  StatusArgs st;
};

// Keys of the order of the scores: NaN above everything, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const unsigned long long u = __double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// Sum over the CTA, for every thread; `buf` alternates between calls.
template <int WARPS>
__device__ __forceinline__ int block_sum(int v, int (&warp_sums)[2][WARPS], int& buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  int* mine = warp_sums[buf ^= 1];
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < WARPS ? mine[threadIdx.x & 31] : 0);
}

// The coefficients of a lane's eight values of a block's bounds: sums over the group's heads of the
// queries' negative parts (lo) or positive parts (hi).
template <typename T>
__device__ __forceinline__ void coefficients(const SelectParams& p, int t, int h, int d0, bool upper, float (&c)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = 0.f;
  const T* q = static_cast<const T*>(p.q) + t * p.q_s0 + int64_t(h) * p.group * p.q_s1 + d0;
  constexpr int kHeads = 4;  // loaded at a time
  for (int g = 0; g < p.group; g += kHeads) {
    uint4 a[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      a[i] = g + i < p.group ? __ldg(reinterpret_cast<const uint4*>(q + (g + i) * p.q_s1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint32_t w[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Pair<T>::values(w[e]);
        // comparisons that let NaN through
        c[2 * e] += upper ? (f.x < 0.f ? 0.f : f.x) : (f.x > 0.f ? 0.f : f.x);
        c[2 * e + 1] += upper ? (f.y < 0.f ? 0.f : f.y) : (f.y > 0.f ? 0.f : f.y);
      }
    }
  }
}

// What a query row sees: its blocks n (0: a row that is out of range), and the place of its request's pages.
struct Row {
  int n, start;
};
__device__ __forceinline__ Row row_of(const SelectParams& p, int b, int pos) {
  Row r{0, 0};
  if (b >= p.batch || pos < 0) return r;
  r.start = __ldg(p.kv_indptr + b);
  const int end = __ldg(p.kv_indptr + b + 1), n = p.page_size.div(pos) + 1;
  if (n <= end - r.start && n <= p.max_blocks) r.n = n;
  return r;
}

// Scores. A round is kTake candidates of a (query, kv head) row: kAhead 16-byte copies per lane, through a ring of the
// warp's own. How many rounds a query has is known on the GPU only, so every CTA adds them up for all queries, and
// each set of up to eight warps, one per kv head, takes an equal run of them: the heads' bounds of a page lie side by
// side and are read at about the same time. (In parts of a fixed length, which short requests leave empty, the same
// loop took 46 us for 64 requests of 2048 to 16384 tokens and 8 kv heads; so it takes 34, of which 5 are the way to
// the first copy, 6.5 TB/s in between.)
struct RoundInfo {
  int row, at, end;  // (query, kv head); candidates [at, end) of it
  uint32_t bits;     // candidates that have a page; kFirst, kLast: round of the row in this run
};
constexpr uint32_t kFirst = 1u << 30, kLast = 1u << 31;

// KEPT: what each query sees is kept from the count of the rounds, for up to kKept queries (64 requests 43.1 against
// 43.7 us, one 18.6 against 19.1, a step of long requests 42.2 against 42.7, in turn and within 0.1). Slices of more
// queries look it up again: 4096 queries of 4096 and 16384 tokens took 101 and 1076 us, in slices of kKept 121 and 1106.
template <typename T, int D, bool KEPT>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kLanes = D / 4;       // lanes of 16 bytes that hold a block's bounds
  constexpr int kPer = 32 / kLanes;   // blocks of one copy instruction
  constexpr int kTake = kAhead * kPer;
  constexpr int kWarps = kScoreThreads / 32;
  extern __shared__ uint4 ring[];
  __shared__ RoundInfo infos[kWarps][kScoreStages];
  // rounds of the queries before each; the place of its request's pages, the blocks that it sees
  __shared__ int warp_sums[kWarps], before[(KEPT ? kKept : kSelectSlice) + 1], starts[KEPT ? kKept : 1];
  __shared__ uint16_t seen[KEPT ? kKept : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();  // the selection's CTAs wait for all of this kernel
  // rounds of each query, added up
  {
    const int per = (p.queries + kScoreThreads - 1) / kScoreThreads;
    const int t0 = min(p.queries, tid * per), t1 = min(p.queries, t0 + per);
    int own = 0;
    for (int t = t0; t < t1; ++t) {
      const int b = __ldg(p.batch_indices + t), pos = __ldg(p.positions + t);
      const Row x = b < 0 ? Row{0, 0} : row_of(p, b, pos);
      before[t] = x.n > p.top_k ? (x.n - p.sink - p.recent + kTake - 1) / kTake : 0;
      if constexpr (KEPT) {
        starts[t] = x.start;
        seen[t] = uint16_t(x.n);
      }
      own += before[t];
    }
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    v += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0) - own;
    for (int t = t0; t < t1; ++t) {
      const int x = before[t];
      before[t] = v;
      v += x;
    }
    if (tid == kScoreThreads - 1) before[p.queries] = v;
    __syncthreads();
  }
  const int per_head = before[p.queries];
  // this warp's set and kv head; the set's run of the rounds of all groups of heads
  const int set = blockIdx.x * p.sets + warp / p.set_heads, h_in = warp % p.set_heads;
  if (warp / p.set_heads >= p.sets) return;
  const int64_t total = int64_t(per_head) * p.head_groups, all = int64_t(gridDim.x) * p.sets;
  int64_t todo = total * set / all;
  const int64_t stop = total * (set + 1) / all;
  const int sub = lane % kLanes, which = lane / kLanes, d0 = 8 * (sub % (D / 8));
  const bool upper = sub >= D / 8;
  uint4* mine = ring + warp * (kScoreStages * kAhead * 32) + lane;

  // What is copied: candidates [at, end) of query t and head h are this run's, pages from `pages` on.
  int t = 0, h = 0, at = 0, end = 0, row_end = 0, window = 0, pg = 0, next_pg = 0;
  uint32_t first = 0;
  const int32_t* pages = nullptr;
  const uint8_t* head = nullptr;
  // lane i: page of candidate at + i (of the last one past the end); looked at when it is needed only, as page 0 with
  // the top bit where there is none
  auto page_at = [&](int i) { return __ldg(pages + min(i + lane, row_end - 1)); };
  auto checked = [&](int x) {
    if (x >= 0 && x < p.num_pages) return x;
    record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    return INT32_MIN;
  };
  auto open = [&]() {
    at = end = 0;
    while (todo < stop) {
      const int group = int(todo / per_head), r = int(todo - int64_t(group) * per_head);
      h = group * p.set_heads + h_in;
      int lo = 0, hi = p.queries;  // the last query whose rounds begin at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= r) lo = mid;
        else hi = mid;
      }
      t = lo;
      const int from = r - before[t], rounds = int(min(int64_t(before[t + 1] - r), stop - todo));
      todo += rounds;
      if (h >= int(p.heads.d)) continue;  // the last group may have fewer heads
      const Row x = KEPT ? Row{seen[t], starts[t]} : row_of(p, __ldg(p.batch_indices + t), __ldg(p.positions + t));
      row_end = x.n - p.sink - p.recent;
      at = from * kTake;
      end = min(row_end, at + rounds * kTake);
      pages = p.kv_indices + x.start + p.sink;
      head = p.bounds + 16 * sub + h * p.b_s1;
      first = kFirst;
      window = at;
      pg = page_at(at);
      next_pg = page_at(at + 32);
      pg = checked(pg);
      return;
    }
  };
  int issued = 0;
  auto issue = [&]() {
    if (at < end) {
      const int stage = issued % kScoreStages;
      if (at - window == 32) {
        window = at;
        pg = checked(next_pg);
        next_pg = page_at(at + 32);
      }
      const int base = at - window;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int from = __shfl_sync(0xffffffffu, pg & INT32_MAX, base + u * kPer + which);
        cp_async_16(mine + (stage * kAhead + u) * 32, head + from * p.b_s0);
      }
      const uint32_t there = (__ballot_sync(0xffffffffu, pg >= 0) >> base) & ((1u << kTake) - 1u);
      const uint32_t bits = there | first | (at + kTake >= end ? kLast : 0u);
      if (lane == 0) infos[warp][stage] = RoundInfo{t * int(p.heads.d) + h, at, min(end, at + kTake), bits};
      first = 0;
      at += kTake;
      ++issued;
      if (at >= end) open();
    }
    cp_async_commit();
  };
  open();
#pragma unroll
  for (int i = 0; i < kScoreStages - 1; ++i) issue();

  float c[8];
  uint32_t largest[4];
  for (int consumed = 0; consumed < issued; ++consumed) {
    __syncwarp();  // the stage that is filled next has been read, and its round is described
    const int stage = consumed % kScoreStages;
    const RoundInfo info = infos[warp][stage];
    issue();
    if (info.bits & kFirst) {
      int head_of;
      const int query = p.heads.divmod(info.row, head_of);
      coefficients<T>(p, query, head_of, d0, upper, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) largest[e] = 0;
    }
    cp_async_wait<kScoreStages - 1>();
    float s[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint4 x = mine[(stage * kAhead + u) * 32];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float2 two = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        two = ffma2(Pair<T>::values(w[e]), make_float2(c[2 * e], c[2 * e + 1]), two);
        largest[e] = Pair<T>::larger(largest[e], w[e]);
      }
      s[u] = two.x + two.y;
    }
    // sums over a block's lanes: halving the blocks a lane holds, then the lanes that hold the same
#pragma unroll
    for (int o = 1, held = kAhead / 2; held >= 1; o <<= 1, held >>= 1) {
#pragma unroll
      for (int u = 0; u < held; ++u) {
        const float send = lane & o ? s[u] : s[u + held];
        const float keep = lane & o ? s[u + held] : s[u];
        s[u] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int o = kAhead; o < kLanes; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    // lane bits 0, 1, 2 chose among 8, 4, 2 blocks: its block is their reversal
    const int u = (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2), i = u * kPer + which;
    if (sub < kAhead && info.at + i < info.end)
      p.scores[int64_t(info.row) * p.stride + info.at + i] = info.bits >> i & 1u ? s[0] : -INFINITY;
    if (info.bits & kLast) {
      // the bound of the sums of absolute products: infinite if any value is, and then the row is scored
      // again
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Pair<T>::values(largest[e]);
        most = fmaf(fabsf(f.x), fabsf(c[2 * e]), most);
        most = fmaf(fabsf(f.y), fabsf(c[2 * e + 1]), most);
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) most += __shfl_xor_sync(0xffffffffu, most, o);
      if (!(most >= 0.f)) most = INFINITY;  // an infinite value times a zero coefficient
      if (kPer > 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
      if (lane == 0) atomicMax(p.most + info.row, __float_as_uint(most));  // bits of numbers above zero are in their order
    }
  }
}

// The scores of a row's m candidates again, where bounds or query values are not finite; every thread of
// the CTA calls it. Of an infinite bound and a coefficient of zero nothing is added; where a head's query
// value is zero, whatever the others' are, its product with an infinite bound is NaN. Returns the bound of the
// sums of absolute products, of the finite bounds. (One request of 131072 tokens, half of its blocks masked,
// takes 133 us where finite ones take 17.3, 64 requests of 16384 133 and 66. As part of the scoring it was 27
// and 110, but finite rows paid: a step took 43.6 instead of 42.1. As a function that is called, the selection
// of 64 finite rows took 44.5 instead of 43.4.)
template <typename T, int D, int THREADS>
__device__ __forceinline__ float score_again(const SelectParams& p, int t, int h, const int32_t* pages,
                                             const uint8_t* head, float* scores, int m) {
  constexpr int kLanes = D / 4, kPer = 32 / kLanes, kWarps = THREADS / 32, kDeep = 4, kStep = kWarps * kPer * kDeep;
  __shared__ float warp_most[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kLanes, which = lane / kLanes, d0 = 8 * (sub % (D / 8));
  float c[8];
  coefficients<T>(p, t, h, d0, sub >= D / 8, c);
  // masks of the halves of pairs of channels: where the coefficient is not zero; where a head's query value is
  uint32_t keep[4], zero[4] = {0, 0, 0, 0}, largest[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) keep[e] = (c[2 * e] != 0.f ? 0xffffu : 0u) | (c[2 * e + 1] != 0.f ? 0xffff0000u : 0u);
  const T* q = static_cast<const T*>(p.q) + t * p.q_s0 + int64_t(h) * p.group * p.q_s1 + d0;
  for (int g = 0; g < p.group; ++g) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(q + g * p.q_s1));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = Pair<T>::values(w[e]);
      zero[e] |= (f.x == 0.f ? 0xffffu : 0u) | (f.y == 0.f ? 0xffff0000u : 0u);
    }
  }
  int pg[kDeep];
  auto look = [&](int i) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) pg[u] = i + u * kPer + which < m ? __ldg(pages + i + u * kPer + which) : -1;
  };
  look(warp * kPer * kDeep);
  for (int i = warp * kPer * kDeep; i < m; i += kStep) {
    uint4 x[kDeep];
    uint32_t there = 0;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const bool ok = pg[u] >= 0 && pg[u] < p.num_pages;
      there |= (ok ? 1u : 0u) << u;
      x[u] = ok ? __ldg(reinterpret_cast<const uint4*>(head + pg[u] * p.b_s0 + 16 * sub)) : make_uint4(0, 0, 0, 0);
    }
    look(i + kStep);
    float s[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float2 two = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t size = w[e] & 0x7fff7fffu, other = Pair<T>::not_infinite(size);
        const uint32_t v = (w[e] & (keep[e] | other)) | (zero[e] & ~other);  // all bits set are NaN
        two = ffma2(Pair<T>::values(v), make_float2(c[2 * e], c[2 * e + 1]), two);
        largest[e] = Pair<T>::larger(largest[e], size & Pair<T>::finite(size));
      }
      s[u] = two.x + two.y;
    }
#pragma unroll
    for (int o = 1, held = kDeep / 2; held >= 1; o <<= 1, held >>= 1) {
#pragma unroll
      for (int u = 0; u < held; ++u) {
        const float send = lane & o ? s[u] : s[u + held];
        const float stay = lane & o ? s[u + held] : s[u];
        s[u] = stay + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int o = kDeep; o < kLanes; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    const int u = (lane & 1) * 2 + ((lane & 2) >> 1), at = i + u * kPer + which;
    if (sub < kDeep && at < m) scores[at] = there >> u & 1u ? s[0] : -INFINITY;
  }
  float most = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = Pair<T>::values(largest[e]);
    most = fmaf(fabsf(f.x), fabsf(c[2 * e]), most);
    most = fmaf(fabsf(f.y), fabsf(c[2 * e + 1]), most);
  }
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) most += __shfl_xor_sync(0xffffffffu, most, o);
  if (!(most >= 0.f)) most = INFINITY;  // a query value is not finite, and no score then is
  if (kPer > 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
  if (lane == 0) warp_most[warp] = most;
  __syncthreads();  // the scores are there too
  most = 0.f;
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, warp_most[w]);
  return most;
}

// Selection: a CTA per (query, kv head) row.
template <typename T, int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kLanes = D / 4, kThreads = THREADS, kWarps = THREADS / 32;
  extern __shared__ __align__(16) uint32_t keys[];  // of the row's candidates, zeros up to a multiple of four; marks
  __shared__ int warp_sums[2][kWarps], part_in[kWarps], part_tie[kWarps];
  __shared__ uint32_t warp_lo[kWarps], warp_hi[kWarps];
  __shared__ int few_at[kFew], few_n, bins[kBins], found_bin, found_n, found_wanted;
  __shared__ uint32_t found_key;
  __shared__ unsigned long long few_key[kFew];
  __shared__ double cd[2 * D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x;
  int h;
  const int t = p.heads.divmod(row, h);
  const int b = __ldg(p.batch_indices + t), pos = __ldg(p.positions + t);
  const Row r = b < 0 ? Row{0, 0} : row_of(p, b, pos);
  // the pages of blocks that are listed without a score, the same for all heads; the scores are still made
  if (h == 0) {
    const int listed = r.n <= p.top_k ? r.n : p.sink + p.recent;
    for (int j = tid; j < listed; j += kThreads) {
      const int pg = __ldg(p.kv_indices + r.start + (r.n <= p.top_k || j < p.sink ? j : r.n - listed + j));
      if (pg < 0 || pg >= p.num_pages) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    }
  }
  wait_for_prior_grid();
  if (b < 0) return;  // a row without a token
  int32_t* out = p.blocks + int64_t(row) * p.top_k;
  const int n = r.n, k = p.top_k - p.sink - p.recent;
  if (n == 0 && tid == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
  if (n <= p.top_k || k == 0) {
    for (int j = tid; j < p.top_k; j += kThreads)
      out[j] = n <= p.top_k ? (j < n ? j : -1) : j < p.sink ? j : n - p.top_k + j;
    return;
  }
  const int m = n - p.sink - p.recent;  // candidates, from block `sink` on
  const int32_t* pages = p.kv_indices + r.start + p.sink;
  float* scores = p.scores + int64_t(row) * p.stride;
  const uint8_t* head = p.bounds + h * p.b_s1;
  const int sub = lane % kLanes;
  const int fours = (m + 3) >> 2;
  float most = __uint_as_float(__ldcg(p.most + row));
  if (!(most < INFINITY)) most = score_again<T, D, THREADS>(p, t, h, pages, head, scores, m);
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = tid; i < fours; i += kAhead * kThreads) {
    float4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u * kThreads < fours) v[u] = __ldcg(reinterpret_cast<const float4*>(scores) + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = 4 * (i + u * kThreads);
      if (at >= m) continue;
      const uint4 x = make_uint4(order_key(v[u].x), at + 1 < m ? order_key(v[u].y) : 0u, at + 2 < m ? order_key(v[u].z) : 0u,
                                 at + 3 < m ? order_key(v[u].w) : 0u);
      reinterpret_cast<uint4*>(keys)[i + u * kThreads] = x;
      lo = min(min(lo, x.x - 1u), min(min(x.y - 1u, x.z - 1u), x.w - 1u));  // keys of scores are above zero
      hi = max(max(hi, x.x), max(max(x.y, x.z), x.w));
    }
  }
  const uint4* keys4 = reinterpret_cast<const uint4*>(keys);
  // kth: the k-th largest key. Keys are counted in 256 bins over their range, then over the bin that holds
  // the k-th, until that has few keys, which are ranked.
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    warp_lo[warp] = lo;
    warp_hi[warp] = hi;
  }
  if (tid < kBins) bins[tid] = 0;
  if (tid == 0) few_n = 0;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? warp_lo[lane] : 0xffffffffu) + 1u;
  hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? warp_hi[lane] : 0u);
  if (tid == 0) p.most[row] = 0;  // every thread has read it; ready for the next run
  int wanted = k;
  uint32_t kth = hi, span = hi - lo;
  for (int shift = max(0, 32 - __clz(hi - lo) - 8);; shift = max(0, shift - 8)) {
    // keys from lo to lo + span by bins
    auto count = [&](uint32_t x) {
      if (x >= lo && x - lo <= span) atomicAdd(&bins[(x - lo) >> shift], 1);
    };
    for (int i = tid; i < fours; i += kThreads) {
      const uint4 x = keys4[i];
      count(x.x);
      count(x.y);
      count(x.z);
      count(x.w);
    }
    __syncthreads();
    // one warp, eight bins a lane: the bins of the lanes before are above
    if (warp == 0) {
      int mine[kBins / 32], sum = 0;
#pragma unroll
      for (int u = 0; u < kBins / 32; ++u) {
        const int at = kBins - 1 - (lane * (kBins / 32) + u);
        sum += mine[u] = bins[at];
        bins[at] = 0;
      }
      int v = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      int before = v - sum;
      if (before < wanted && wanted <= v) {
#pragma unroll
        for (int u = 0; u < kBins / 32; ++u) {
          if (before < wanted && wanted <= before + mine[u]) {
            found_bin = kBins - 1 - (lane * (kBins / 32) + u);
            found_n = mine[u];
            found_wanted = wanted - before;
          }
          before += mine[u];
        }
      }
    }
    __syncthreads();
    lo += uint32_t(found_bin) << shift;
    span = (1u << shift) - 1;
    wanted = found_wanted;
    if (shift == 0) {
      kth = lo;
      break;
    }
    if (found_n <= kFew) {
      for (int i = tid; i < m; i += kThreads)
        if (keys[i] >= lo && keys[i] - lo <= span) few_at[atomicAdd(&few_n, 1)] = int(keys[i]);
      __syncthreads();
      if (tid < found_n) {
        const uint32_t x = uint32_t(few_at[tid]);
        int larger = 0, same = 0;
        for (int j = 0; j < found_n; ++j) {
          larger += uint32_t(few_at[j]) > x;
          same += uint32_t(few_at[j]) == x;
        }
        if (larger < wanted && wanted <= larger + same) found_key = x;
      }
      __syncthreads();
      kth = found_key;
      break;
    }
  }
  int buf = 0;
  // certain above key_hi, out below key_lo
  uint32_t key_lo = kth, key_hi = kth;
  const float threshold = key_value(kth);
  // products below fp32's normal numbers are off by half of their least step each (none is where all are zero)
  const float err = most > 0.f ? most * p.error + 7.2e-43f : 0.f;
  if (kth != 0xffffffffu && fabsf(threshold) < INFINITY) {
    key_hi = order_key(__fadd_ru(threshold, 2.f * err));
    key_lo = order_key(__fadd_rd(threshold, -2.f * err));
  }
  int counts = 0;  // keys above key_hi, and in the upper half word those from key_lo on: both below 2^16
  static_assert(kSelectMaxBlocks < 1 << 16, "two counts in a word");
  for (int i = tid; i < fours; i += kThreads) {
    const uint4 x = keys4[i];
    counts += (x.x > key_hi) + (x.y > key_hi) + (x.z > key_hi) + (x.w > key_hi);
    counts += ((x.x >= key_lo) + (x.y >= key_lo) + (x.z >= key_lo) + (x.w >= key_lo)) << 16;
  }
  if (tid == 0) few_n = 0;
  counts = block_sum(counts, warp_sums, buf);
  const int above = counts & 0xffff, between = int(unsigned(counts) >> 16) - above;
  const int want = k - above;  // of those between
  // Candidates stay whose key is above `sure`, and of those with the key `tie` the first `rest`.
  uint32_t sure = key_hi, tie = key_lo;
  int rest = want;
  if (between == want) {
    sure = key_lo - 1;  // key_lo is above 0: it is the key of a number, or NaN's
    rest = 0;
  } else if (key_lo != key_hi) {
    // fp64 scores of the blocks between, with coefficients that the CTA adds up once: fp64 is slow here
    for (int i = tid; i < 2 * D; i += kThreads) {
      const T* q = static_cast<const T*>(p.q) + t * p.q_s0 + int64_t(h) * p.group * p.q_s1 + i % D;
      double sum = 0.0;
#pragma unroll 4
      for (int g = 0; g < p.group; ++g) {
        const float x = to_float(q[g * p.q_s1]);
        sum += double(i >= D ? (x < 0.f ? 0.f : x) : (x > 0.f ? 0.f : x));
      }
      cd[i] = sum;
    }
    __syncthreads();
    const double* mine = cd + 8 * sub;
    auto score64 = [&](int i) {
      const int pg = __ldg(pages + i);
      double s = -INFINITY;
      if (pg >= 0 && pg < p.num_pages) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(head + pg * p.b_s0 + 16 * sub));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        s = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Pair<T>::values(w[e]);
          // times zero: a score that fp32 can order has no infinite bound's product
          s = mine[2 * e] != 0.0 ? fma(double(f.x), mine[2 * e], s) : s;
          s = mine[2 * e + 1] != 0.0 ? fma(double(f.y), mine[2 * e + 1], s) : s;
        }
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return order_key(s);
    };
    // They are marked in place: chosen ones above every number's key, equal ones of which only the
    // first are with key_hi, others below.
    rest = 0;
    tie = key_hi;
    if (between <= kFew) {
      for (int i = tid; i < m; i += kThreads)
        if (keys[i] >= key_lo && keys[i] <= key_hi) few_at[atomicAdd(&few_n, 1)] = i;
      __syncthreads();
      for (int j = warp; j < between; j += kWarps) {
        const unsigned long long key = score64(few_at[j]);
        if (lane == 0) few_key[j] = key;
      }
      __syncthreads();
      if (tid < between) {
        int rank = 0;
        for (int j = 0; j < between; ++j)
          rank += few_key[j] > few_key[tid] || (few_key[j] == few_key[tid] && few_at[j] < few_at[tid]);
        keys[few_at[tid]] = rank < want ? 0xffffffffu : 0u;
      }
    } else {
      // the fp64 keys' halves take the places of the fp32 scores and of their keys; a bit marks each
      uint32_t *marks = keys + p.stride, *upper = reinterpret_cast<uint32_t*>(scores);
      for (int i = warp * 32; i < m; i += kThreads) {
        const uint32_t key = i + lane < m ? keys[i + lane] : 0u;
        const uint32_t mark = __ballot_sync(0xffffffffu, key >= key_lo && key <= key_hi);
        if (lane == 0) marks[i >> 5] = mark;
        for (uint32_t todo = mark; todo; todo &= todo - 1) {
          const int at = i + __ffs(todo) - 1;
          const unsigned long long k64 = score64(at);
          if (lane == 0) {
            upper[at] = uint32_t(k64 >> 32);
            keys[at] = uint32_t(k64);
          }
        }
      }
      __syncthreads();
      auto marked = [&](int i) { return (marks[i >> 5] >> (i & 31) & 1u) != 0; };
      auto exact = [&](int i) { return (unsigned long long)(upper[i]) << 32 | keys[i]; };
      auto count = [&](unsigned long long from) {
        int cnt = 0;
        for (int i = tid; i < m; i += kThreads) cnt += marked(i) && exact(i) >= from;
        return block_sum(cnt, warp_sums, buf);
      };
      unsigned long long kth64 = 0;
      for (int bit = 63; bit >= 0; --bit)
        if (count(kth64 | (1ull << bit)) >= want) kth64 |= 1ull << bit;
      rest = want - (kth64 == ~0ull ? 0 : count(kth64 + 1));
      for (int i = tid; i < m; i += kThreads)
        if (marked(i)) keys[i] = exact(i) > kth64 ? 0xffffffffu : exact(i) == kth64 ? key_hi : 0u;
    }
    __syncthreads();
  }

  // each warp writes a contiguous run of the candidates, four of them a lane: counts, then places
  const int run = ((fours + kWarps - 1) / kWarps + 31) & ~31;
  const int r0 = min(fours, warp * run), r1 = min(fours, r0 + run);
  const bool has_ties = rest > 0;
  int in = 0, ties = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint4 x = keys4[i];
    in += (x.x > sure) + (x.y > sure) + (x.z > sure) + (x.w > sure);
    if (has_ties) ties += (x.x == tie) + (x.y == tie) + (x.z == tie) + (x.w == tie);
  }
  in = __reduce_add_sync(0xffffffffu, in);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    part_in[warp] = in;
    part_tie[warp] = ties;
  }
  __syncthreads();
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? part_in[lane] : 0);
  int eq = __reduce_add_sync(0xffffffffu, lane < warp ? part_tie[lane] : 0);
  at += p.sink + min(eq, rest);
  const uint32_t below = (1u << lane) - 1;
  for (int i = r0 + lane; i - lane < r1; i += 32) {
    const uint4 x4 = i < r1 ? keys4[i] : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
    bool stay[4];
    int rank = eq;  // ties before this lane's
    if (has_ties) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t lanes = __ballot_sync(0xffffffffu, x[u] == tie);
        rank += __popc(lanes & below);
        eq += __popc(lanes);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      stay[u] = x[u] > sure || (has_ties && x[u] == tie && rank < rest);
      rank += x[u] == tie;
    }
    if (!__any_sync(0xffffffffu, stay[0] || stay[1] || stay[2] || stay[3])) continue;
    int to = at;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t lanes = __ballot_sync(0xffffffffu, stay[u]);
      to += __popc(lanes & below);
      at += __popc(lanes);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (stay[u]) out[to++] = p.sink + 4 * i + u;
  }
  for (int j = tid; j < p.sink; j += kThreads) out[j] = j;
  for (int j = tid; j < p.recent; j += kThreads) out[p.top_k - p.recent + j] = n - p.recent + j;
}

bskv_status check_bounds(const char* who, const void* bounds, const int64_t* strides, int32_t head_dim) {
  if (!bounds || !strides || !aligned16(bounds)) { set_error("%s: bounds must be a 16-byte aligned tensor", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i)
    if (strides[i] < 2 * head_dim || strides[i] % 8) {
      set_error("%s: bounds stride %d (%lld elements) must be a multiple of 16 bytes, at least one head's bounds", who, i, (long long)strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  return BSKV_OK;
}

template <typename T, int D, int THREADS>
bskv_status launch_select(const SelectParams& p, int64_t rows, bool scored, cudaStream_t st) {
  auto kern = select_kernel<T, D, THREADS>;
  static std::atomic<int> allowed[64];
  const size_t smem = sizeof(uint32_t) * (size_t(p.stride) + (size_t(p.stride) + 31) / 32);
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "run_select_blocks: cudaFuncSetAttribute")) return s;
  // it may begin while the scores are made, and waits for them
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(rows));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = scored ? 1 : 0;
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, p), "run_select_blocks launch");
}

// Slices of at most `slice` queries, one after the other: the scores of all of them share the workspace.
template <typename T, int D>
bskv_status launch_both(SelectParams p, int64_t queries, int64_t slice, int num_sms, cudaStream_t st) {
  constexpr int kWarps = kScoreThreads / 32;
  const bool kept = std::min(queries, slice) <= kKept;
  auto kern = kept ? score_kernel<T, D, true> : score_kernel<T, D, false>;
  static std::atomic<int> allowed[2][64];
  constexpr size_t smem = size_t(kWarps) * kScoreStages * kAhead * 32 * sizeof(uint4);
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed[kept], "run_select_blocks: cudaFuncSetAttribute")) return s;
  const int heads = int(p.heads.d);
  p.set_heads = std::min(heads, kWarps);
  p.sets = kWarps / p.set_heads;
  p.head_groups = (heads + p.set_heads - 1) / p.set_heads;
  for (int64_t t0 = 0; t0 < queries; t0 += slice) {
    p.queries = int(std::min(slice, queries - t0));
    const bool scored = p.max_blocks > p.top_k && p.top_k > p.sink + p.recent;  // else there is no choice
    if (scored) {
      // rounds that there may be: a set of warps has some of them
      const int64_t rounds = (int64_t(p.max_blocks) + 7) / 8 * p.queries * p.head_groups;
      const int grid = int(std::min<int64_t>((rounds + p.sets - 1) / p.sets, int64_t(kScoreCtas) * num_sms));
      kern<<<unsigned(grid), kScoreThreads, smem, st>>>(p);
      if (bskv_status s = cuda_check(cudaGetLastError(), "run_select_blocks score launch")) return s;
    }
    const int64_t rows = int64_t(p.queries) * heads;
    const auto launch = p.max_blocks > kSelectWide ? launch_select<T, D, 1024> : launch_select<T, D, 256>;
    if (bskv_status s = launch(p, rows, scored, st)) return s;
    p.q = static_cast<const T*>(p.q) + slice * p.q_s0;
    p.batch_indices += slice;
    p.positions += slice;
    p.blocks += slice * heads * p.top_k;
  }
  return BSKV_OK;
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_block_bounds_paged(
    const void* kv_cache, const int64_t* kv_strides, int32_t dtype, int32_t num_kv_heads,
    int32_t head_dim, int32_t page_size, int64_t num_pages, const int32_t* batch_indices,
    const int32_t* positions, int64_t nnz, const int32_t* kv_indptr, const int32_t* kv_indices,
    const int32_t* kv_last_page_len, int32_t batch, void* bounds, const int64_t* bounds_strides,
    void* stream) {
  BSKV_NVTX_RANGE("bskv_block_bounds_paged");
  const char* who = "block_bounds_paged";
  if (dtype != BSKV_BF16 && dtype != BSKV_FP16) { set_error("%s: dtype %s unsupported", who, dtype_name(dtype)); return BSKV_ERR_UNSUPPORTED; }
  if (head_dim != 64 && head_dim != 128) { set_error("%s: head_dim %d not in {64,128}", who, head_dim); return BSKV_ERR_UNSUPPORTED; }
  if (num_kv_heads < 1 || page_size < 1 || num_pages < 0 || nnz < 0 || batch < 0) {
    set_error("%s: num_kv_heads=%d page_size=%d num_pages=%lld nnz=%lld batch=%d", who, num_kv_heads, page_size,
              (long long)num_pages, (long long)nnz, batch);
    return BSKV_ERR_INVALID_ARG;
  }
  if (num_pages > INT32_MAX) { set_error("%s: num_pages=%lld", who, (long long)num_pages); return BSKV_ERR_UNSUPPORTED; }
  if (nnz == 0) return BSKV_OK;
  if (!batch_indices || !positions || !kv_indptr || !kv_indices || !kv_last_page_len) { set_error("%s: NULL argument", who); return BSKV_ERR_INVALID_ARG; }
  if (!kv_cache || !kv_strides || !aligned16(kv_cache)) { set_error("%s: kv_cache must be a 16-byte aligned tensor", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 4; ++i)
    if (kv_strides[i] <= 0 || kv_strides[i] % 8) {
      set_error("%s: kv stride %d (%lld elements) must be positive and 16-byte aligned", who, i, (long long)kv_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  if (bskv_status s = check_bounds(who, bounds, bounds_strides, head_dim)) return s;
  BoundsParams p{};
  p.keys = static_cast<const uint8_t*>(kv_cache);
  p.k_s0 = 2 * kv_strides[0]; p.k_s2 = 2 * kv_strides[2]; p.k_s3 = 2 * kv_strides[3];
  p.bounds = static_cast<uint8_t*>(bounds); p.b_s0 = 2 * bounds_strides[0]; p.b_s1 = 2 * bounds_strides[1];
  p.batch_indices = batch_indices; p.positions = positions;
  p.kv_indptr = kv_indptr; p.kv_indices = kv_indices; p.kv_last_page_len = kv_last_page_len;
  p.nnz = nnz; p.heads = num_kv_heads; p.batch = batch; p.num_pages = int(num_pages);
  p.page_size = FastDiv(page_size);
  // a row at a time while the GPU has a warp for each row and head, up to a warp's lanes of them
  constexpr int kWarps = kBoundsThreads / 32, kSms = 152;
  const int64_t warps = int64_t(kSms) * kBoundsCtas * kWarps;
  p.rows = int(std::min<int64_t>(kBoundsRows, (nnz * num_kv_heads + warps - 1) / warps));
  const int64_t units = (nnz + p.rows - 1) / p.rows * num_kv_heads;
  if (units > INT32_MAX / 2) { set_error("%s: too many rows", who); return BSKV_ERR_UNSUPPORTED; }
  p.units = int(units);
  p.by_head = FastDiv(num_kv_heads);
  if (bskv_status s = status_args(&p.st)) return s;
  const unsigned grid = unsigned(std::min<int64_t>((units + kWarps - 1) / kWarps, int64_t(kSms) * kBoundsCtas));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto kern = head_dim == 128 ? (dtype == BSKV_BF16 ? bounds_kernel<__nv_bfloat16, 128> : bounds_kernel<__half, 128>)
                              : (dtype == BSKV_BF16 ? bounds_kernel<__nv_bfloat16, 64> : bounds_kernel<__half, 64>);
  constexpr size_t smem = size_t(kWarps) * kBoundsStages * kBoundsAhead * 32 * sizeof(uint4);
  static std::atomic<int> allowed[4][64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed[(head_dim == 128) * 2 + (dtype == BSKV_BF16)], "block_bounds_paged: cudaFuncSetAttribute"))
    return s;
  kern<<<grid, kBoundsThreads, smem, st>>>(p);
  return cuda_check(cudaGetLastError(), "block_bounds_paged launch");
}

extern "C" bskv_status bskv_run_select_blocks(
    const bskv_plan* plan, const void* q, const int64_t* q_strides, const void* bounds,
    const int64_t* bounds_strides, const int32_t* batch_indices, const int32_t* positions,
    const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch, int32_t* blocks,
    void* float_ws, size_t float_ws_bytes, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_select_blocks");
  const char* who = "run_select_blocks";
  if (bskv_status s = check_blocks_run(who, plan, batch_indices, positions, kv_indptr, kv_indices, batch, blocks, float_ws, float_ws_bytes)) return s;
  if (plan->M == 0) return BSKV_OK;
  if (!q || !q_strides || !aligned16(q)) { set_error("%s: q must be a 16-byte aligned tensor", who); return BSKV_ERR_INVALID_ARG; }
  if (plan->num_pages == 0) { set_error("%s: a cache without pages", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] < 0 || q_strides[i] % 8) {
      set_error("%s: q stride %d (%lld elements) must be a multiple of 16 bytes", who, i, (long long)q_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  if (bskv_status s = check_bounds(who, bounds, bounds_strides, plan->head_dim)) return s;
  const BlocksWorkspace ws = blocks_workspace(plan);
  uint8_t* base = static_cast<uint8_t*>(float_ws);
  SelectParams p{};
  p.q = q; p.q_s0 = q_strides[0]; p.q_s1 = q_strides[1];
  p.bounds = static_cast<const uint8_t*>(bounds); p.b_s0 = 2 * bounds_strides[0]; p.b_s1 = 2 * bounds_strides[1];
  p.batch_indices = batch_indices; p.positions = positions; p.kv_indptr = kv_indptr; p.kv_indices = kv_indices;
  p.blocks = blocks;
  p.scores = reinterpret_cast<float*>(base + ws.scores);
  p.most = reinterpret_cast<unsigned*>(plan->counters_dev);
  p.group = plan->num_qo_heads / plan->num_kv_heads;
  p.batch = batch; p.num_pages = plan->num_pages; p.max_blocks = plan->max_blocks; p.stride = ws.stride;
  p.top_k = plan->top_k; p.sink = plan->sink; p.recent = plan->recent;
  p.page_size = FastDiv(plan->page_size); p.heads = FastDiv(plan->num_kv_heads);
  p.error = float((p.group + 10) * 1.01 * std::ldexp(1.0, -24));
  if (bskv_status s = status_args(&p.st)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = plan->dtype == BSKV_BF16;
  const auto launch = plan->head_dim == 128 ? (bf16 ? launch_both<__nv_bfloat16, 128> : launch_both<__half, 128>)
                                            : (bf16 ? launch_both<__nv_bfloat16, 64> : launch_both<__half, 64>);
  return launch(p, plan->M, ws.slice, plan->num_sms, st);
}
