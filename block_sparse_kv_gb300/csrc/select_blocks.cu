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
// can do per byte, so scoring is bound by reading the bounds once.
//
// Selection. The first `sink` and the last `recent` blocks that a query sees stay, and of the others the k of
// highest score, as 64-bit arithmetic would choose them (the lowest index among equals). Scores are summed in
// fp32 with an error of at most E = (group + 16) 2^-24 max_j sum_d |hi_d P_d| + |lo_d N_d|: coefficients
// are sums of up to `group` terms, a lane's eight products one chain, five more additions join the lanes.
// With s_k the k-th largest fp32 score, blocks above s_k + 2 E are chosen and those below s_k - 2 E are
// not, whatever the rounding; only the blocks between are scored again, in fp64. Rows where nothing lies
// between but as many blocks as are still wanted (nearly all) need no second look.
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
constexpr int kBoundsRows = 32;  // most token rows that a CTA looks at

struct BoundsParams {
  const uint8_t* keys;
  int64_t k_s0, k_s2, k_s3;  // bytes: page, kv head, slot
  uint8_t* bounds;
  int64_t b_s0, b_s1;        // bytes: page, kv head
  const int32_t *batch_indices, *positions, *kv_indptr, *kv_indices, *kv_last_page_len;
  int64_t nnz;
  int heads, batch, num_pages, rows;
  FastDiv page_size;
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
  static __device__ __forceinline__ float2 values(uint32_t a) {
    return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
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
  static __device__ __forceinline__ float2 values(uint32_t a) {
    return __half22float2(*reinterpret_cast<const __half2*>(&a));
  }
};

// A CTA looks at `rows` token rows, a warp takes kv heads in turn. A page is done for each row that is
// its first among consecutive rows: in whatever order the rows are, the lowest position of a page
// is one of those, and a page that is done twice gets the same bytes. (Bound by reading the keys: rows
// are D / 8 lanes of 16 bytes, eight of them in flight per lane.)
template <typename T, int D>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kLanes = D / 8, kSlots = 32 / kLanes, kAhead = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = int64_t(blockIdx.x) * p.rows;
  // lane i: row first + i
  int page = -1, fill = 0;
  if (lane < p.rows && first + lane < p.nnz) {
    const int64_t i = first + lane;
    const int b = __ldg(p.batch_indices + i), pos = __ldg(p.positions + i);
    int slot = 0;
    const int j = pos >= 0 ? p.page_size.divmod(pos, slot) : 0;
    const bool before = i > 0 && __ldg(p.batch_indices + i - 1) == b && __ldg(p.positions + i - 1) == pos - 1;
    if (b >= 0 && (slot == 0 || !before || pos < 0)) {
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
  const uint32_t todo = __ballot_sync(0xffffffffu, page >= 0);
  const int sub = lane % kLanes, slot0 = lane / kLanes;
  for (uint32_t m = todo; m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    const int pg = __shfl_sync(0xffffffffu, page, src), n = __shfl_sync(0xffffffffu, fill, src);
    for (int h = warp; h < p.heads; h += kBoundsThreads / 32) {
      const uint8_t* from = p.keys + pg * p.k_s0 + h * p.k_s2 + slot0 * p.k_s3 + 16 * sub;
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = Pair<T>::kInf;
        hi[c] = Pair<T>::kNegInf;
      }
      for (int s = 0; s < n; s += kSlots * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (s + i * kSlots + slot0 < n) x[i] = __ldg(reinterpret_cast<const uint4*>(from + int64_t(s + i * kSlots) * p.k_s3));
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (s + i * kSlots + slot0 >= n) continue;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            lo[c] = Pair<T>::low(lo[c], w[c]);
            hi[c] = Pair<T>::high(hi[c], w[c]);
          }
        }
      }
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          lo[c] = Pair<T>::low(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], o));
          hi[c] = Pair<T>::high(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], o));
        }
      }
      // lo, then hi: 2 kLanes lanes write
      if (lane < 2 * kLanes) {
        const bool upper = lane >= kLanes;
        *reinterpret_cast<uint4*>(p.bounds + pg * p.b_s0 + h * p.b_s1 + 16 * lane) =
            upper ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------------------

constexpr int kThreads = kSelectThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 8;    // loads that a lane has in flight
constexpr int kFew = 32;     // blocks between the bounds of certainty that are ranked by one warp

struct SelectParams {
  const void* q;
  int64_t q_s0, q_s1;
  const uint8_t* bounds;
  int64_t b_s0, b_s1;  // bytes: page, kv head
  const int32_t *batch_indices, *positions, *kv_indptr, *kv_indices;
  int32_t* blocks;
  float* scores;               // [rows][max_blocks]
  float* sums;                 // [rows][parts]: largest sums of absolute products
  unsigned long long* exact;   // [rows][max_blocks]: keys of fp64 scores
  int* counters;               // [rows]
  int group, batch, num_pages, max_blocks, parts, top_k, sink, recent;
  FastDiv page_size, heads, by_parts;
  float error;                 // E over the sum of absolute products
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

// Sum over the CTA, for every thread; `buf` alternates between calls.
__device__ __forceinline__ int block_sum(int v, int (&warp_sums)[2][kWarps], int& buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  int* mine = warp_sums[buf ^= 1];
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += mine[w];
  return s;
}

// The coefficients of a lane's eight values of a block's bounds: sums over the group's heads of the
// queries' negative parts (lo) or positive parts (hi).
template <typename T, typename F>
__device__ __forceinline__ void coefficients(const SelectParams& p, int t, int h, int d0, bool upper, F (&c)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = F(0);
  const T* q = static_cast<const T*>(p.q) + t * p.q_s0 + int64_t(h) * p.group * p.q_s1 + d0;
  for (int g = 0; g < p.group; ++g) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(q + g * p.q_s1));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = Pair<T>::values(w[e]);
      // comparisons that let NaN through
      c[2 * e] += F(upper ? (f.x < 0.f ? 0.f : f.x) : (f.x > 0.f ? 0.f : f.x));
      c[2 * e + 1] += F(upper ? (f.y < 0.f ? 0.f : f.y) : (f.y > 0.f ? 0.f : f.y));
    }
  }
}

// One part of a (query, kv head) row's blocks is scored by each of its CTAs; the last one to finish
// selects.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kLanes = D / 4;       // lanes of 16 bytes that hold a block's bounds
  constexpr int kPer = 32 / kLanes;   // blocks of one load instruction
  extern __shared__ uint32_t keys[];  // of the row's candidates
  __shared__ int warp_sums[2][kWarps], part_in[kWarps], part_tie[kWarps];
  __shared__ float warp_most[kWarps];
  __shared__ uint32_t warp_lo[kWarps], warp_hi[kWarps];
  __shared__ int few_at[kFew], few_n, is_last;
  __shared__ unsigned long long few_key[kFew];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int part;
  const int row = p.by_parts.divmod(blockIdx.x, part);
  int h;
  const int t = p.heads.divmod(row, h);
  const int b = __ldg(p.batch_indices + t);
  if (b < 0) return;  // a row without a token
  const int pos = __ldg(p.positions + t);
  int32_t* out = p.blocks + int64_t(row) * p.top_k;
  bool bad = b >= p.batch || pos < 0;
  int start = 0, n = 0;
  if (!bad) {
    start = __ldg(p.kv_indptr + b);
    n = p.page_size.div(pos) + 1;
    bad = n > __ldg(p.kv_indptr + b + 1) - start || n > p.max_blocks;
  }
  if (bad) {
    if (part == 0 && tid == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    n = 0;
  }
  const int k = p.top_k - p.sink - p.recent;
  if (n <= p.top_k || k == 0) {
    if (part == 0) {
      for (int j = tid; j < p.top_k; j += kThreads)
        out[j] = n <= p.top_k ? (j < n ? j : -1) : j < p.sink ? j : n - p.top_k + j;
    }
    return;
  }
  const int m = n - p.sink - p.recent;  // candidates, from block `sink` on
  const int32_t* pages = p.kv_indices + start + p.sink;
  // parts of whole rounds of the CTA's warps
  constexpr int kRound = kWarps * kAhead * kPer;
  const int share = ((m + p.parts - 1) / p.parts + kRound - 1) / kRound * kRound;
  const int active = (m + share - 1) / share;
  if (part >= active) return;
  const int i0 = part * share, i1 = min(m, i0 + share);
  float* scores = p.scores + int64_t(row) * p.max_blocks;
  const uint8_t* head = p.bounds + h * p.b_s1;
  const int sub = lane % kLanes, which = lane / kLanes, d0 = 8 * (sub % (D / 8));
  const bool upper = sub >= D / 8;

  float c[8];
  coefficients<T, float>(p, t, h, d0, upper, c);
  float most = 0.f;
  for (int i = i0 + warp * kAhead * kPer; i < i1; i += kRound) {
    // lane u: page of candidate i + u
    int pg = -1;
    if (lane < kAhead * kPer && i + lane < i1) {
      pg = __ldg(pages + i + lane);
      if (pg < 0 || pg >= p.num_pages) {
        record_error(p.st, BSKV_ERR_DEVICE_INDEX);
        pg = -1;
      }
    }
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int from = __shfl_sync(0xffffffffu, pg, u * kPer + which);
      x[u] = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(head + from * p.b_s0 + 16 * sub)) : make_uint4(0, 0, 0, 0);
    }
    float s[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float a = 0.f;
      s[u] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Pair<T>::values(w[e]);
        s[u] = fmaf(f.x, c[2 * e], s[u]);
        a = fmaf(fabsf(f.x), fabsf(c[2 * e]), a);
        s[u] = fmaf(f.y, c[2 * e + 1], s[u]);
        a = fmaf(fabsf(f.y), fabsf(c[2 * e + 1]), a);
      }
      // an infinite or NaN score has no rounding
      most = a < INFINITY ? fmaxf(most, a) : most;
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
    const int u = (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2);
    const int at = u * kPer + which;
    const bool there = __shfl_sync(0xffffffffu, pg, at) >= 0;
    if (sub < kAhead && i + at < i1) {
      const float v = there ? s[0] : -INFINITY;
      if (active == 1) keys[i + at] = order_key(v);
      else scores[i + at] = v;
    }
  }
  // sums of absolute products: over the lanes of the largest
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) most += __shfl_xor_sync(0xffffffffu, most, o);
  most = kPer == 1 ? most : fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
  if (lane == 0) warp_most[warp] = most;
  __syncthreads();
  most = warp_most[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) most = fmaxf(most, warp_most[w]);
  if (active > 1) {
    float* sums = p.sums + int64_t(row) * p.parts;
    if (tid == 0) {
      sums[part] = most;
      const int old = atomic_add_acq_rel(p.counters + row, 1);  // releases what the CTA wrote before the barrier
      is_last = old == active - 1;
    }
    __syncthreads();
    if (!is_last) return;
    for (int i = tid; i < m; i += kThreads) keys[i] = order_key(__ldcg(scores + i));
    for (int i = 0; i < active; ++i) most = fmaxf(most, __ldcg(sums + i));
    if (tid == 0) p.counters[row] = 0;  // ready for the next run
    __syncthreads();
  }

  // kth: the k-th largest key, bit by bit below the bits that all keys share
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = tid; i < m; i += kThreads) {
    lo = min(lo, keys[i]);
    hi = max(hi, keys[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    warp_lo[warp] = lo;
    warp_hi[warp] = hi;
  }
  if (tid == 0) few_n = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo, warp_lo[w]);
    hi = max(hi, warp_hi[w]);
  }
  int buf = 0;
  uint32_t kth = lo;
  if (lo != hi) {
    const int top = 31 - __clz(lo ^ hi);
    kth = hi >> top >> 1 << top << 1;  // two shifts: `top` may be 31
    for (int bit = top; bit >= 0; --bit) {
      const uint32_t cand = kth | (1u << bit);
      int cnt = 0;
      for (int i = tid; i < m; i += kThreads) cnt += keys[i] >= cand;
      cnt = block_sum(cnt, warp_sums, buf);
      if (cnt >= k) kth = cand;
      if (cnt == k) break;
    }
    // exactly k keys from here on: the k-th is the lowest of them
    uint32_t least = 0xffffffffu;
    for (int i = tid; i < m; i += kThreads)
      if (keys[i] >= kth) least = min(least, keys[i]);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) warp_lo[warp] = least;
    __syncthreads();
    kth = warp_lo[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) kth = min(kth, warp_lo[w]);
  }
  // certain above key_hi, out below key_lo
  uint32_t key_lo = kth, key_hi = kth;
  const float threshold = key_value(kth);
  const float err = most * p.error;
  if (kth != 0xffffffffu && fabsf(threshold) < INFINITY) {
    key_hi = order_key(__fadd_ru(threshold, 2.f * err));
    key_lo = order_key(__fadd_rd(threshold, -2.f * err));
  }
  int above = 0, between = 0;
  for (int i = tid; i < m; i += kThreads) {
    above += keys[i] > key_hi;
    between += keys[i] >= key_lo && keys[i] <= key_hi;
  }
  above = block_sum(above, warp_sums, buf);
  between = block_sum(between, warp_sums, buf);
  const int want = k - above;  // of those between
  // Candidates stay whose key is above `sure`, and of those with the key `tie` the first `rest`.
  uint32_t sure = key_hi, tie = key_lo;
  int rest = want;
  if (between == want) {
    sure = key_lo - 1;  // key_lo is above 0: it is the key of a number, or NaN's
    rest = 0;
  } else if (key_lo != key_hi) {
    // fp64 scores of the blocks between
    double cd[8];
    coefficients<T, double>(p, t, h, d0, upper, cd);
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
          s = fma(double(f.x), cd[2 * e], s);
          s = fma(double(f.y), cd[2 * e + 1], s);
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
      unsigned long long* exact = p.exact + int64_t(row) * p.max_blocks;
      for (int i = warp * 32; i < m; i += kThreads) {
        const uint32_t key = i + lane < m ? keys[i + lane] : 0u;
        for (uint32_t todo = __ballot_sync(0xffffffffu, key >= key_lo && key <= key_hi); todo; todo &= todo - 1) {
          const int at = i + __ffs(todo) - 1;
          const unsigned long long k64 = score64(at);
          if (lane == 0) exact[at] = k64;
        }
      }
      __syncthreads();
      auto count = [&](unsigned long long from) {
        int cnt = 0;
        for (int i = tid; i < m; i += kThreads)
          cnt += keys[i] >= key_lo && keys[i] <= key_hi && exact[i] >= from;
        return block_sum(cnt, warp_sums, buf);
      };
      unsigned long long kth64 = 0;
      for (int bit = 63; bit >= 0; --bit)
        if (count(kth64 | (1ull << bit)) >= want) kth64 |= 1ull << bit;
      rest = want - (kth64 == ~0ull ? 0 : count(kth64 + 1));
      for (int i = tid; i < m; i += kThreads)
        if (keys[i] >= key_lo && keys[i] <= key_hi) keys[i] = exact[i] > kth64 ? 0xffffffffu : exact[i] == kth64 ? key_hi : 0u;
    }
    __syncthreads();
  }

  // each warp writes a contiguous run of the candidates: counts, then places
  const int run = ((m + kWarps - 1) / kWarps + 31) & ~31;
  const int r0 = min(m, warp * run), r1 = min(m, r0 + run);
  int in = 0, ties = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    in += keys[i] > sure;
    ties += rest > 0 && keys[i] == tie;
  }
  in = __reduce_add_sync(0xffffffffu, in);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    part_in[warp] = in;
    part_tie[warp] = ties;
  }
  __syncthreads();
  int at = 0, eq = 0;
  for (int w = 0; w < warp; ++w) {
    at += part_in[w];
    eq += part_tie[w];
  }
  at += p.sink + min(eq, rest);
  const uint32_t below = (1u << lane) - 1;
  for (int i = r0 + lane; i - lane < r1; i += 32) {
    const uint32_t key = i < r1 ? keys[i] : 0u;
    const bool tied = i < r1 && rest > 0 && key == tie;
    const uint32_t tied_lanes = __ballot_sync(0xffffffffu, tied);
    const bool stay = (i < r1 && key > sure) || (tied && eq + __popc(tied_lanes & below) < rest);
    eq += __popc(tied_lanes);
    const uint32_t staying = __ballot_sync(0xffffffffu, stay);
    if (stay) out[at + __popc(staying & below)] = p.sink + i;
    at += __popc(staying);
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

template <typename T, int D>
bskv_status launch_select(const SelectParams& p, int64_t rows, cudaStream_t st) {
  auto kern = select_kernel<T, D>;
  static std::atomic<int> allowed[64];
  const size_t smem = sizeof(uint32_t) * size_t(p.max_blocks);
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "run_select_blocks: cudaFuncSetAttribute")) return s;
  kern<<<unsigned(rows * p.parts), kThreads, smem, st>>>(p);
  return cuda_check(cudaGetLastError(), "run_select_blocks launch");
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
  // a row per CTA while there are fewer rows than keep the GPU busy, up to a warp's lanes of them
  p.rows = int(std::min<int64_t>(kBoundsRows, (nnz + 1215) / 1216));
  if ((nnz + p.rows - 1) / p.rows > INT32_MAX) { set_error("%s: too many rows", who); return BSKV_ERR_UNSUPPORTED; }
  if (bskv_status s = status_args(&p.st)) return s;
  const unsigned grid = unsigned((nnz + p.rows - 1) / p.rows);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) {
    if (dtype == BSKV_BF16) bounds_kernel<__nv_bfloat16, 128><<<grid, kBoundsThreads, 0, st>>>(p);
    else bounds_kernel<__half, 128><<<grid, kBoundsThreads, 0, st>>>(p);
  } else {
    if (dtype == BSKV_BF16) bounds_kernel<__nv_bfloat16, 64><<<grid, kBoundsThreads, 0, st>>>(p);
    else bounds_kernel<__half, 64><<<grid, kBoundsThreads, 0, st>>>(p);
  }
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
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] < 0 || q_strides[i] % 8) { set_error("%s: q stride %d (%lld elements) must be a multiple of 16 bytes", who, i, (long long)q_strides[i]); return BSKV_ERR_INVALID_ARG; }
  if (bskv_status s = check_bounds(who, bounds, bounds_strides, plan->head_dim)) return s;
  const int64_t rows = int64_t(plan->M) * plan->num_kv_heads;
  const BlocksWorkspace ws = blocks_workspace(plan);
  uint8_t* base = static_cast<uint8_t*>(float_ws);
  SelectParams p{};
  p.q = q; p.q_s0 = q_strides[0]; p.q_s1 = q_strides[1];
  p.bounds = static_cast<const uint8_t*>(bounds); p.b_s0 = 2 * bounds_strides[0]; p.b_s1 = 2 * bounds_strides[1];
  p.batch_indices = batch_indices; p.positions = positions; p.kv_indptr = kv_indptr; p.kv_indices = kv_indices;
  p.blocks = blocks;
  p.exact = reinterpret_cast<unsigned long long*>(base + ws.exact);
  p.scores = reinterpret_cast<float*>(base + ws.scores);
  p.sums = reinterpret_cast<float*>(base + ws.sums);
  p.counters = plan->counters_dev;
  p.group = plan->num_qo_heads / plan->num_kv_heads;
  p.batch = batch; p.num_pages = plan->num_pages; p.max_blocks = plan->max_blocks; p.parts = ws.parts;
  p.top_k = plan->top_k; p.sink = plan->sink; p.recent = plan->recent;
  p.page_size = FastDiv(plan->page_size); p.heads = FastDiv(plan->num_kv_heads); p.by_parts = FastDiv(ws.parts);
  p.error = float((p.group + 16) * 1.01 * std::ldexp(1.0, -24));
  if (bskv_status s = status_args(&p.st)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (plan->head_dim == 128)
    return plan->dtype == BSKV_BF16 ? launch_select<__nv_bfloat16, 128>(p, rows, st) : launch_select<__half, 128>(p, rows, st);
  return plan->dtype == BSKV_BF16 ? launch_select<__nv_bfloat16, 64>(p, rows, st) : launch_select<__half, 64>(p, rows, st);
}
