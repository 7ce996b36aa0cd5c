// Accumulated attention weight per cached token: the scores that eviction goes by.
//
// Mathematics. For every key j of request b and kv head h
//   w_j = sum over the queries t of b that see j, and the query heads r of h's group, of
//         exp(scale q_tr . k_j - lse_tr)
//   score_j <- (j new ? 0 : decay score_j) + w_j
// With the log-sum-exp known (the attention run returned it) a weight needs K and the query
// only, each key's sum is independent of every other's, and one warp makes it: no atomics, and
// the same bits on every run.
//
// Two kernels, by the query rows (queries times heads of the group) of the longest request:
//   * stream (up to 16 rows, the decode step): keys are the M = 16 rows of mma.sync m16n8k16, query
//     rows its N = 8 columns, so a key's sum stays in its lanes until one reduction over the four
//     lanes of its row. A row's lane reads 16-byte chunks t, t + 4, ...: products of chunk c with the
//     same chunk of the query are two k-steps, whatever the order of the dims. Query fragments stay
//     in registers, each warp streams a range of tokens through a private ring of 32-token tiles
//     filled by 16-byte asynchronous copies. Bound by reading K: 64 requests of 512 to 4096 tokens
//     in 16 bits 52.0 us (6.0 TB/s); in 4 bits by instructions: 8 of 32000 to 40000 36.6 us (4.8 TB/s).
//   * tile (more rows, a prefill window): S = K Q^T by tcgen05, 128 keys against up to 128 query rows
//     a product. A key is a TMEM lane and so a thread, which reads its row of S and adds up its
//     weights: no reduction between threads, and two packed FMAs and two exponentials per two
//     weights. The last 32 queries of 16 prompts, 128 rows, take 41.5 us (4.3 TB/s; 32 rows 32.3 us): no pipe is full,
//     each item waits for its keys, its product and its columns of tensor memory.
// 4-bit keys (E2M1 codes times 2^x per 32 values): the stream kernel multiplies codes and f16
// queries and scales each block's fp32 partial sum; the tile kernel turns a key once into the
// query's type, relative to its largest scale, and multiplies that back after the product.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "cache_common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.h"
#include "page_walk.cuh"

namespace bskv {
namespace {

using namespace dev;

constexpr int kStages = 3;
constexpr int kTile = kWalkTile;     // tokens per stage of the stream kernel
constexpr int kWarps = kWeightsWarps;
constexpr int kKeys = kWeightsKeys;  // keys per CTA of the tile kernel, one per computing thread
constexpr int kPanel = kKeys * 128;  // 128 rows of 64 16-bit values, swizzled

struct WeightsParams {
  const int32_t* meta;
  const void* q;
  int64_t q_s0, q_s1;
  const uint8_t* keys;              // 16-bit keys or codes
  int64_t k_s0, k_s1, k_s2, k_s3;   // bytes: page, K/V, kv head, slot
  const uint8_t* scales;            // 4-bit keys
  int64_t s_s0, s_s2;               // bytes
  const float* lse;
  float* scores;
  int64_t w_s0, w_s1;               // floats: page, kv head
  int num_kv_heads, group, num_qo_heads, causal;
  FastDiv heads, groups, page_size, queries;
  int box, tile_queries, num_items, num_requests;  // tile kernel: keys per TMA box, queries per product
  int single;                                      // no item has more than one product
  int off_workers, off_records, off_aux1, off_req, num_workers;
  int take;                                        // stream kernel: workers per warp
  float decay, scale_log2;
  StatusArgs st;
};

// The request's queries, in the metadata: first row of q, number of queries, tokens.
struct Request {
  int qo, nq, len;
};
__device__ __forceinline__ Request request_of(const WeightsParams& p, int b) {
  const int32_t* r = p.meta + p.off_req + 3 * b;
  return Request{__ldg(r), __ldg(r + 1), __ldg(r + 2)};
}

// A query row's part of the exponent and its factor: exp(x - lse) = exp2(x log2e - hi) r with
// hi + log2(1 / r) = lse log2e to about 48 bits, so that rounding lse log2e to fp32 costs the
// weight nothing. Rows that add nothing (no query there, or one that saw no key) have last = -1,
// the last key that a row sees.
struct RowInfo {
  float hi, r;
  int last;
};
__device__ __forceinline__ RowInfo row_info(const WeightsParams& p, const Request& rq, float lse, int tok) {
  RowInfo o{0.f, 0.f, -1};
  if (lse == -INFINITY) return o;
  constexpr float kLog2eLow = 1.925963033500011e-8f;  // log2 e - fp32(log2 e)
  o.hi = lse * kLog2e;
  const float lo = isinf(o.hi) ? 0.f : fmaf(lse, kLog2e, -o.hi) + lse * kLog2eLow;
  o.r = exp2f(-lo);
  o.last = p.causal ? tok + rq.len - rq.nq : rq.len - 1;
  return o;
}
// Log-sum-exp of query row `row` (token, head of the group); -inf past the request's queries.
__device__ __forceinline__ float row_lse(const WeightsParams& p, const Request& rq, int kvh, int row) {
  int head;
  const int t = p.groups.divmod(row, head);
  if (t >= rq.nq) return -INFINITY;
  return __ldg(p.lse + int64_t(rq.qo + t) * p.num_qo_heads + kvh * p.group + head);
}

// Sums over the four lanes of a quad: lane t gets that of x[t].
__device__ __forceinline__ float quad_sums(const float (&x)[4], int t) {
  const float a = (t & 2 ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, t & 2 ? x[0] : x[2], 2);
  const float b = (t & 2 ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, t & 2 ? x[1] : x[3], 2);
  return (t & 1 ? b : a) + __shfl_xor_sync(0xffffffffu, t & 1 ? a : b, 1);
}

// ---------------------------------------------------------------------------------------
// stream kernel
// ---------------------------------------------------------------------------------------

template <int D, bool FP4>
struct Shape {
  static constexpr int kBlocks = D / kFp4Block;
  static constexpr int kRow = FP4 ? D / 2 : 2 * D;
  static constexpr int kParts = kRow / 16;
  static constexpr int kScales = kTile * kRow;                          // stage offsets
  static constexpr int kOld = kScales + (FP4 ? kTile * kBlocks : 0);    // scores read
  static constexpr int kPlace = kOld + 4 * kTile;                       // where they belong
  static constexpr int kStage = kPlace + 8 * (kTile / 8);
  static constexpr int kRing = kStages * ((kStage + 127) / 128 * 128);
  // What the copy of rows kRows i .. of a group adds to addresses by XOR, as part() stores them.
  static __device__ __forceinline__ constexpr int turn(int i) { return FP4 ? i << 4 : (i & 1) << 6; }
  // Stored part of part c of row r: word and 16-byte reads of the compute loop then fall into
  // distinct banks.
  static __device__ __forceinline__ int part(int r, int c) {
    if constexpr (FP4) return c ^ ((r >> (D == 128 ? 1 : 2)) & (kParts - 1));
    else return c ^ ((r & 1) << 2);
  }
};

// The query rows of a unit in B-operand order, with their exponents. Column j of a lane is row
// 8 (j / 2) + 2 t + (j & 1).
template <int D, int NT>
struct Rows {
  uint32_t q[NT][D / 32][4];
  float c[2 * NT];
  RowInfo info[2 * NT];
};

template <typename T, int D, int NT, bool FP4>
__device__ __forceinline__ void load_rows(const WeightsParams& p, const Request& rq, int kvh, int lane,
                                          Rows<D, NT>& s) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * nt + g, tok = p.groups.div(row);
    const bool live = tok < rq.nq;
    const T* src = static_cast<const T*>(p.q) + int64_t(rq.qo + tok) * p.q_s0 +
                   (int64_t(kvh) * p.group + (row - tok * p.group)) * p.q_s1;
    float back = 1.f;
    if constexpr (FP4) {
      back = load_q_f16<T, D / 32>(src, live, false, lane, s.q[nt]);
    } else {
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * t)) : make_uint4(0, 0, 0, 0);
        s.q[nt][j][0] = x.x;
        s.q[nt][j][1] = x.y;
        s.q[nt][j][2] = x.z;
        s.q[nt][j][3] = x.w;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s.c[2 * nt + e] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t + 4 * e);
      const int r = 8 * nt + 2 * t + e;
      s.info[2 * nt + e] = row_info(p, rq, row_lse(p, rq, kvh, r), p.groups.div(r));
    }
  }
}

// q . k of 16 keys (rows 16 h + g and + 8 of the tile) with the unit's rows, in fp32.
template <typename T, int D, int NT, bool FP4>
__device__ __forceinline__ void dot_tile(const uint8_t* st, int h, int lane, const Rows<D, NT>& s,
                                         float (&x)[NT][4]) {
  using Sh = Shape<D, FP4>;
  const int g = lane >> 2, t = lane & 3, r0 = 16 * h + g, r1 = r0 + 8;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
  if constexpr (FP4) {
    float s0[D / 32], s1[D / 32];
    scales_of<D / 32>(scale_word<D>(st + Sh::kScales, r0), s0);
    scales_of<D / 32>(scale_word<D>(st + Sh::kScales, r1), s1);
#pragma unroll
    for (int blk = 0; blk < D / 32; ++blk) {
      uint32_t a0[4], a1[4];
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(st + r0 * Sh::kRow + (Sh::part(r0, blk) << 4) + 4 * t), a0);
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(st + r1 * Sh::kRow + (Sh::part(r1, blk) << 4) + 4 * t), a1);
      const uint32_t f0[4] = {a0[0], a1[0], a0[1], a1[1]}, f1[4] = {a0[2], a1[2], a0[3], a1[3]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        MmaOp<__half>::run(acc, f0, s.q[nt][blk][0], s.q[nt][blk][1]);
        MmaOp<__half>::run(acc, f1, s.q[nt][blk][2], s.q[nt][blk][3]);
        x[nt][0] = fmaf(acc[0], s0[blk], x[nt][0]);
        x[nt][1] = fmaf(acc[1], s0[blk], x[nt][1]);
        x[nt][2] = fmaf(acc[2], s1[blk], x[nt][2]);
        x[nt][3] = fmaf(acc[3], s1[blk], x[nt][3]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint4 a0 = *reinterpret_cast<const uint4*>(st + r0 * Sh::kRow + (Sh::part(r0, t + 4 * j) << 4));
      const uint4 a1 = *reinterpret_cast<const uint4*>(st + r1 * Sh::kRow + (Sh::part(r1, t + 4 * j) << 4));
      const uint32_t f0[4] = {a0.x, a1.x, a0.y, a1.y}, f1[4] = {a0.z, a1.z, a0.w, a1.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        MmaOp<T>::run(x[nt], f0, s.q[nt][j][0], s.q[nt][j][1]);
        MmaOp<T>::run(x[nt], f1, s.q[nt][j][2], s.q[nt][j][3]);
      }
    }
  }
}

template <typename T, int D, int NT, bool FP4>
__global__ void __launch_bounds__(kWarps * 32, weights_ctas_per_sm(D, FP4))
    weights_stream_kernel(const WeightsParams p) {
  using Sh = Shape<D, FP4>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kStride = Sh::kRing / kStages;
  uint8_t* ring = smem + warp * Sh::kRing;
  const int w = (blockIdx.x * kWarps + warp) * p.take;
  if (w >= p.num_workers) return;
  const int c0 = __ldg(p.meta + p.off_workers + w);
  const int nck = __ldg(p.meta + p.off_workers + min(w + p.take, p.num_workers)) - c0;
  const int32_t* records = p.meta + p.off_records + c0 * kWalkWords;
  PageWalk walk(records, nck, p.meta + p.off_aux1, p.heads, p.page_size, lane);
  const bool old = p.decay != 0.f;

  // Eight lanes copy a group of 8 tokens: 16-byte parts of rows, then one or two pieces of the
  // scales, two of the scores, and where these belong. What the addresses add to the group's own
  // offset, kept by lane (tok - win) / 8 + j, is fixed.
  const int j = lane >> 3, sub = lane & 7;
  constexpr int kLanes = Sh::kParts < 8 ? Sh::kParts : 8;  // side by side in a row
  constexpr int kRows = 8 / kLanes;                        // rows a copy instruction covers
  constexpr int kPieces = 8 * Sh::kBlocks / 16;
  const int row = sub / kLanes;
  const uint8_t* k_lane = p.keys + row * p.k_s3 + sub % kLanes * 16;
  const int64_t step = kRows * p.k_s3;
  const uint32_t to_lane = smem_u32(ring + (8 * j + row) * Sh::kRow + sub % kLanes * 16);
  const bool takes_scales = FP4 && sub < kPieces, takes_scores = old && (sub & 6) == 4;
  const uint32_t scales_to = smem_u32(ring + Sh::kScales + 8 * j * Sh::kBlocks + sub * 16);
  const uint32_t scores_to = smem_u32(ring + Sh::kOld + 32 * j + (sub & 1) * 16);
  int64_t k_off = 0, s_off = 0, w_off = 0;
  auto issue = [&](int stage) {
    if (walk.live()) {
      if (walk.enter()) {
        k_off = walk.page * p.k_s0 + walk.kvh * p.k_s2 + walk.slot * p.k_s3;
        if constexpr (FP4) s_off = walk.page * p.s_s0 + walk.kvh * p.s_s2 + walk.slot * Sh::kBlocks;
        w_off = walk.page * p.w_s0 + walk.kvh * p.w_s1 + walk.slot;
      }
      const uint8_t* from = k_lane + walk.of_group(k_off, 8 * j);
      const uint8_t* s_from = FP4 ? p.scales + walk.of_group(s_off, 8 * j) + sub * 16 : nullptr;
      const int64_t place = walk.of_group(w_off, 8 * j);
      if (walk.has(8 * j)) {
        const uint32_t at = stage * kStride;
#pragma unroll
        for (int i = 0; i < 8 / kRows; ++i) {
#pragma unroll
          for (int c = 0; c < Sh::kParts; c += kLanes)
            cp_async_16_at(((to_lane + at) ^ Sh::turn(i)) + i * kRows * Sh::kRow + 16 * c, from + 16 * c);
          from += step;
        }
        if (takes_scales) cp_async_16_at(scales_to + at, s_from);
        if (takes_scores) cp_async_16_at(scores_to + at, p.scores + place + 4 * (sub & 1));
        if (sub == 0) *reinterpret_cast<int64_t*>(ring + at + Sh::kPlace + 8 * j) = place;
      }
      walk.advance();
    }
    cp_async_commit();
  };
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  const int g = lane >> 2, t = lane & 3;
  Rows<D, NT> s;
  int done = 0;
  for (int k = 0; k < nck; ++k) {
    const WalkChunk ch = walk_chunk(records, k);
    int kvh;
    const int b = p.heads.divmod(ch.unit, kvh);
    const Request rq = request_of(p, b);
    load_rows<T, D, NT, FP4>(p, rq, kvh, lane, s);
    // tiles up to here are seen by all rows, are whole and of older tokens
    int plain = min(ch.end, rq.len - rq.nq);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
      if (s.info[j].last >= 0) plain = min(plain, s.info[j].last + 1);
    plain = __reduce_min_sync(0xffffffffu, plain);
    for (int at = ch.begin; at < ch.end; at += kTile, ++done) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // the tile is there for every lane, and the stage refilled next is free
      issue((done + kStages - 1) % kStages);
      const uint8_t* st = ring + (done % kStages) * kStride;
      auto tile = [&](auto is_plain) {
        float sum[4];  // keys at + 8 i + g
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[NT][4];
          dot_tile<T, D, NT, FP4>(st, h, lane, s, x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = at + 16 * h + 8 * i + g;
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * NT; ++j) {
              const float e = fast_exp2(fmaf(x[j >> 1][2 * i + (j & 1)], s.c[j], -s.info[j].hi));
              if (is_plain ? s.info[j].last >= 0 : key <= s.info[j].last) a = fmaf(e, s.info[j].r, a);
            }
            sum[2 * h + i] = a;
          }
        }
        // lane (g, t) writes key at + 8 t + g
        const float mine = quad_sums(sum, t);
        const int r = 8 * t + g;
        if (is_plain || at + r < ch.end) {
          float* dst = p.scores + *reinterpret_cast<const int64_t*>(st + Sh::kPlace + 8 * t) + g;
          const bool fresh = !old || (!is_plain && at + r >= rq.len - rq.nq);
          *dst = fresh ? mine : fmaf(p.decay, *reinterpret_cast<const float*>(st + Sh::kOld + 4 * r), mine);
        }
      };
      if (at + kTile <= plain) tile(std::true_type{});
      else tile(std::false_type{});
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------------------
// tile kernel
// ---------------------------------------------------------------------------------------

// 16 bytes (8 values) of a 4-bit key as a chunk of T, in units of the row's largest scale; f a power of
// two, at most 1.
template <typename T>
__device__ __forceinline__ uint4 widen(uint32_t w, float f) {
  uint32_t h[4], o[4];
  cvt_e2m1x8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 x = *reinterpret_cast<__half2*>(&h[i]);
    if constexpr (__is_same(T, __half)) {  // below 2^-24 of the largest block a value may round
      x = __hmul2(x, __float2half2_rn(f));
      o[i] = *reinterpret_cast<uint32_t*>(&x);
    } else {
      const float2 a = __half22float2(x);
      o[i] = MmaOp<T>::pack(a.x * f, a.y * f);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct TileShared {
  float4 pair[2][2][64];  // [group of threads][parity] of query rows 2 i and 2 i + 1: {-hi, -hi, r, r}
  int last[2][2][128];
  float part[2][kKeys];   // the second group's sums of an item
  float unit[4][kKeys];   // 4-bit keys: what a key's products are multiplied by
  uint64_t k_full[2], k_empty[2], q_full[2], q_empty[2], s_full[2], s_empty[2];
  uint32_t tmem;
  int abort;
};

// An item of the tile kernel: 128 keys of a request for one kv head. Items are numbered by request,
// head, then keys, and a CTA takes a contiguous range: its queries mostly stay the same.
struct TileItem {
  int r, kvh, c;              // request record, kv head, which 128 keys
  int begin, end, pbase, tok0, tiles;
  Request rq;
  int tiles_of_keys;          // of the request
};
// Record of request r of the plan: {first item, 128-key tiles, tokens, kv_indptr, first query, queries}.
__device__ __forceinline__ void place_item(const WeightsParams& p, TileItem& t) {
  t.begin = t.c * kKeys;
  t.end = min(t.begin + kKeys, t.rq.len);
  // causal: the first query that sees the first key
  t.tok0 = p.causal ? max(0, t.begin - (t.rq.len - t.rq.nq)) : 0;
  t.tiles = t.tok0 < t.rq.nq ? p.queries.div(t.rq.nq - t.tok0 + p.tile_queries - 1) : 0;
}
__device__ __forceinline__ void open_request(const WeightsParams& p, TileItem& t) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p.meta + p.off_records) + 2 * t.r);
  const int4 q = __ldg(reinterpret_cast<const int4*>(p.meta + p.off_records) + 2 * t.r + 1);
  t.tiles_of_keys = a.y;
  t.pbase = a.w;
  t.rq = Request{q.x, q.y, a.z};
}
// By the whole warp: 32 records at a time, for the last whose first item is at most i.
__device__ __forceinline__ TileItem find_item(const WeightsParams& p, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int n = p.num_requests; n > 1;) {
    const int step = (n + 31) >> 5, at = lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, at < n && __ldg(p.meta + p.off_records + kWalkWords * (lo + at)) <= i);
    const int k = (31 - __clz(m)) * step;
    lo += k;
    n = min(step, n - k);
  }
  TileItem t;
  t.r = lo;
  open_request(p, t);
  const int rest = i - __ldg(p.meta + p.off_records + kWalkWords * lo);
  t.kvh = rest / t.tiles_of_keys;
  t.c = rest - t.kvh * t.tiles_of_keys;
  place_item(p, t);
  return t;
}
// The item after t, which exists.
__device__ __forceinline__ TileItem next_item(const WeightsParams& p, TileItem t) {
  if (++t.c == t.tiles_of_keys) {
    t.c = 0;
    if (++t.kvh == p.num_kv_heads) {
      t.kvh = 0;
      ++t.r;
      open_request(p, t);
    }
  }
  place_item(p, t);
  return t;
}

// Two groups of a thread per key, a warp that copies and multiplies, and for 4-bit keys a group that
// turns them into 16 bits.
constexpr int tile_threads(bool fp4) { return (fp4 ? 3 : 2) * kKeys + 32; }

// A 4-bit key's row and scales on their way to shared memory.
template <int D>
struct Row4 {
  uint4 w[D / 32];
  uint32_t code[D / 32];
};

// Products alternate between two TMEM buffers, each with a group of 128 threads that adds up its
// weights, so that one group's exponentials run under the other's waits. Two modes:
//   * single: no request has more query rows than one product takes. Item n of the CTA goes to group
//     n mod 2; keys have two buffers too, queries stay while they are the same.
//   * several products per item: they alternate between the groups, whose sums are added at its end;
//     queries have two buffers, keys one.
template <typename T, int D, bool FP4>
__global__ void __launch_bounds__(tile_threads(FP4), 2)
    weights_tile_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ WeightsParams p) {
  constexpr int kPanels = D / 64;
  constexpr uint32_t kBuffer = uint32_t(kPanels * kPanel), kTmem = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ks = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const bool single = p.single;
  uint8_t* qs = ks + (single ? 2 : 1) * kBuffer;
  TileShared& sh = *reinterpret_cast<TileShared*>(ks + 3 * kBuffer);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], FP4 ? kKeys : 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], FP4 ? 2 : 1);
      mbar_init(&sh.s_empty[i], kKeys);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&sh.tmem, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const bool forced = forced_timeout(p.st);
  volatile int* abort_flag = &sh.abort;
  const int i0 = int(int64_t(blockIdx.x) * p.num_items / gridDim.x);
  const int i1 = int(int64_t(blockIdx.x + 1) * p.num_items / gridDim.x);
  TileItem t = find_item(p, i0);

  if (warp == 8) {
    // The warp stays converged; one lane's copies and products are executed. The next item's keys
    // are copied before this item's product where they have a buffer of their own.
    const uint32_t leader = elect_leader();
    bool ok = true;
    const uint64_t once = l2_evict_first_policy(), again = l2_evict_last_policy();
    const uint32_t fmt = __is_same(T, __half) ? 0u : 1u;
    const uint32_t idesc = umma_idesc(128, uint32_t((p.tile_queries * p.group + 15) & ~15), fmt, fmt, 0, 0);
    const uint64_t dk = umma_desc(smem_u32(ks), 16, 1024, kSwz128), dq = umma_desc(smem_u32(qs), 16, 1024, kSwz128);
    TileItem next = i0 + 1 < i1 ? next_item(p, t) : t;
    int page = 0, slot = 0;  // of the lane's box of the item whose keys are copied next
    auto lookup = [&](const TileItem& u) {
      const int key = u.begin + lane * p.box;  // at most 16 boxes
      if (!FP4 && u.tiles > 0 && lane * p.box < kKeys && key < u.end)
        page = __ldg(p.meta + p.off_aux1 + u.pbase + p.page_size.divmod(key, slot));
    };
    // Times each buffer was filled (keys, queries) or multiplied into (products).
    int kn0 = 0, kn1 = 0, qn = 0, sn0 = 0, sn1 = 0;
    auto wait = [&](uint64_t* bar, int phase) { return issuer_wait(bar, uint32_t(phase) & 1u, p.st, forced, abort_flag); };
    auto load_k = [&](const TileItem& u, int kb) {
      if (u.tiles == 0) return true;
      int& n = kb ? kn1 : kn0;
      if constexpr (!FP4) {
        if (n > 0 && !wait(&sh.k_empty[kb], n - 1)) return false;
        const int boxes = (u.end - u.begin + p.box - 1) / p.box;
        mbar_arrive_expect_tx_w(leader, &sh.k_full[kb], uint32_t(boxes) * kPanels * p.box * 128);
        for (int x = 0; x < boxes; ++x) {
          const int pg = __shfl_sync(0xffffffffu, page, x), sl = __shfl_sync(0xffffffffu, slot, x);
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn)
            tma_load_5d_hint_w(leader, ks + kb * kBuffer + pn * kPanel + x * p.box * 128, &kmap, pn * 64, sl, u.kvh, 0,
                               pg, &sh.k_full[kb], once);
        }
      }
      ++n;
      return true;
    };
    auto load_q = [&](int tok, int qb) {
      mbar_arrive_expect_tx_w(leader, &sh.q_full[qb], uint32_t(kPanels) * p.tile_queries * p.group * 128);
#pragma unroll
      for (int pn = 0; pn < kPanels; ++pn)
        tma_load_3d_hint_w(leader, qs + qb * kBuffer + pn * kPanel, &qmap, pn * 64, t.kvh * p.group, t.rq.qo + tok,
                           &sh.q_full[qb], again);
      ++qn;
    };
    auto multiply = [&](int kb, int qb, int sb, bool last) {
      int& n = sb ? sn1 : sn0;
      if (n > 0 && !wait(&sh.s_empty[sb], n - 1)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
        umma_f16_w(leader, tmem + sb * 128, dk + ((kb * kBuffer) >> 4) + at, dq + ((qb * kBuffer) >> 4) + at, idesc,
                   kk > 0 ? 1u : 0u);
      }
      umma_commit_w(leader, &sh.s_full[sb]);
      if constexpr (FP4) {  // with an arrival of its own the warp hands on the units that k_full gave it
        if (leader) mbar_arrive(&sh.s_full[sb]);
        __syncwarp();
      }
      if (!single) umma_commit_w(leader, &sh.q_empty[qb]);
      if (last) umma_commit_w(leader, &sh.k_empty[kb]);
      ++n;
      return true;
    };
    int q_r = -1, q_h = -1, q_tok = -1;  // single: whose queries are in the buffer
    int prev = 0;                        // and the buffer of the last product
    lookup(t);
    ok = load_k(t, 0);
    for (int i = i0; i < i1 && ok; ++i) {
      const TileItem after = i + 2 < i1 ? next_item(p, next) : next;
      const bool more = i + 1 < i1;
      const int par = (i - i0) & 1;
      if (single) {
        if (more) lookup(next);
        if (t.tiles > 0 && (t.r != q_r || t.kvh != q_h || t.tok0 != q_tok)) {
          // the one buffer: the products that read the old queries are done first
          const int n = prev ? sn1 : sn0;
          ok = n == 0 || wait(&sh.s_full[prev], n - 1);
          if (!ok) break;
          load_q(t.tok0, 0);
          q_r = t.r;
          q_h = t.kvh;
          q_tok = t.tok0;
        }
        if (more) ok = load_k(next, par ^ 1);
        if (ok && t.tiles > 0) {
          ok = wait(&sh.k_full[par], (par ? kn1 : kn0) - 1) && wait(&sh.q_full[0], qn - 1) && multiply(par, 0, par, true);
          prev = par;
        }
      } else {
        int q = 0;  // query tiles of the item copied
        const int q0 = qn;
        auto fill = [&]() {
          const int qb = qn & 1;
          if (qn >= 2 && !wait(&sh.q_empty[qb], (qn >> 1) - 1)) return false;
          load_q(t.tok0 + q * p.tile_queries, qb);
          ++q;
          return true;
        };
        while (ok && q < 2 && q < t.tiles) ok = fill();
        if (ok && t.tiles > 0) ok = wait(&sh.k_full[0], kn0 - 1);
        for (int n = 0; n < t.tiles && ok; ++n) {
          const int u = q0 + n;  // query tiles and products are numbered alike
          ok = wait(&sh.q_full[u & 1], u >> 1) && multiply(0, u & 1, u & 1, n == t.tiles - 1);
          if (ok && q < t.tiles) ok = fill();
        }
        if (more && ok) {
          lookup(next);
          ok = load_k(next, 0);
        }
      }
      t = next;
      next = after;
    }
    if (!ok) {
      // copies and products in flight land before the CTA leaves (bounded, not forcible)
      *abort_flag = 1;
      if (sn0 > 0) mbar_wait(&sh.s_full[0], uint32_t(sn0 - 1) & 1u, p.st, false);
      if (sn1 > 0) mbar_wait(&sh.s_full[1], uint32_t(sn1 - 1) & 1u, p.st, false);
      if (!FP4 && kn0 > 0) mbar_wait(&sh.k_full[0], uint32_t(kn0 - 1) & 1u, p.st, false);
      if (!FP4 && kn1 > 0) mbar_wait(&sh.k_full[1], uint32_t(kn1 - 1) & 1u, p.st, false);
      for (int n = max(0, qn - (single ? 1 : 2)); n < qn; ++n)
        mbar_wait(&sh.q_full[single ? 0 : n & 1], uint32_t(single ? n : n >> 1) & 1u, p.st, false);
    }
  } else if (FP4 && warp > 8) {
    // A thread per key turns 4-bit rows into 16 bits; the next item's row is read ahead.
    const int tid = threadIdx.x - (2 * kKeys + 32);
    auto read_row = [&](const TileItem& u, int page) {
      Row4<D> x{};
      const int key = u.begin + tid;
      int sl;
      p.page_size.divmod(key, sl);
      if (u.tiles > 0 && key < u.end) {
        const uint8_t* src = p.keys + page * p.k_s0 + u.kvh * p.k_s2 + sl * p.k_s3;
        const uint8_t* sc = p.scales + page * p.s_s0 + u.kvh * p.s_s2 + sl * (D / 32);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          x.w[j] = __ldg(reinterpret_cast<const uint4*>(src) + j);
          x.code[j] = __ldg(sc + j);
        }
      }
      return x;
    };
    // The row as T relative to its largest scale into key buffer kb; its products' unit. A slot of
    // units is written again when the products that use it have been read: two fills of a buffer on
    // (single: a buffer's products belong to one group), or four (several: they alternate, and a fill
    // has one product at least).
    auto put_row = [&](const Row4<D>& x, int kb, int slot) {
      uint32_t top = 0;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        bad = bad || x.code[j] == 255u;
        // a block of zeros does not count, whatever its scale
        if ((x.w[j].x | x.w[j].y | x.w[j].z | x.w[j].w) & 0x77777777u) top = max(top, x.code[j]);
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int d = min(0, int(x.code[j]) - int(top));  // above 0 only for zeros
        const float f = d < -126 ? 0.f : pow2(d);
        const uint32_t v[4] = {x.w[j].x, x.w[j].y, x.w[j].z, x.w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sts128(smem_u32(ks) + (kb * kPanels + (j >> 1)) * kPanel + swz(tid, (j & 1) * 4 + i, 128), widen<T>(v[i], f));
      }
      sh.unit[slot][tid] = bad ? NAN : p.scale_log2 * e8m0_value(top);
      fence_proxy_async_smem();
      mbar_arrive(&sh.k_full[kb]);
    };

    auto page_of = [&](const TileItem& u) {
      const int key = u.begin + tid;
      return key < u.end ? __ldg(p.meta + p.off_aux1 + u.pbase + p.page_size.div(key)) : 0;
    };
    int kn0 = 0, kn1 = 0;  // fills of the buffers
    TileItem next = i0 + 1 < i1 ? next_item(p, t) : t;
    Row4<D> row = read_row(t, page_of(t));
    int page = page_of(next);
    for (int i = i0; i < i1; ++i) {
      const Row4<D> ahead = read_row(next, page);
      const TileItem after = i + 2 < i1 ? next_item(p, next) : next;
      page = page_of(after);
      if (t.tiles > 0) {
        const int kb = single ? (i - i0) & 1 : 0;
        int& n = kb ? kn1 : kn0;
        if (n > 0 && !warp_wait(&sh.k_empty[kb], uint32_t(n - 1) & 1u, p.st, forced, abort_flag)) {
          if (lane == 0) *abort_flag = 1;
          break;
        }
        put_row(row, kb, single ? 2 * kb + (n & 1) : n & 3);
        ++n;
      }
      row = ahead;
      t = next;
      next = after;
    }
  } else {
    // What an item needs from memory is read an item ahead: the page of the thread's key, the key's
    // score and the log-sum-exps.
    const int grp = warp >> 2, tid = threadIdx.x & (kKeys - 1), bar = 1 + grp;
    const uint32_t row = tmem + (uint32_t(warp & 3) << 21) + grp * 128;  // TMEM lane 32 * (warp mod 4)
    int my_head;
    const int my_tok = p.groups.divmod(tid, my_head);  // of query row tid of a product
    auto page_of = [&](const TileItem& u) {
      const int key = u.begin + tid;
      return key < u.end ? __ldg(p.meta + p.off_aux1 + u.pbase + p.page_size.div(key)) : 0;
    };
    auto score_at = [&](const TileItem& u, int page) {
      int slot;
      p.page_size.divmod(u.begin + tid, slot);
      return p.scores + page * p.w_s0 + u.kvh * p.w_s1 + slot;
    };
    auto is_fresh = [&](const TileItem& u) { return p.decay == 0.f || u.begin + tid >= u.rq.len - u.rq.nq; };
    auto old_score = [&](const TileItem& u, const float* at) {
      return u.begin + tid < u.end && !is_fresh(u) ? __ldg(at) : 0.f;
    };
    auto lse_of = [&](const TileItem& u, int n) {  // of row tid of product n
      const int tok = u.tok0 + n * p.tile_queries + my_tok;
      if (n >= u.tiles || my_tok >= p.tile_queries || tok >= u.rq.nq) return -INFINITY;
      return __ldg(p.lse + int64_t(u.rq.qo + tok) * p.num_qo_heads + u.kvh * p.group + my_head);
    };
    bool ok = true;
    int sn = 0;        // products of this group so far
    int products = 0, fills = 0;  // several: of the CTA, and key tiles
    float2 sum[2];
    // The group's weights of one product of item u (query tokens from tok on), lse its row's.
    auto add_weights = [&](const TileItem& u, int tok, float lse) {
      const int info = sn & 1, key = u.begin + tid;
      const int count = min(p.tile_queries, u.rq.nq - tok) * p.group;
      const RowInfo o = row_info(p, u.rq, lse, tok + my_tok);
      sh.last[grp][info][tid] = o.last;
      float* pair = reinterpret_cast<float*>(&sh.pair[grp][info][tid >> 1]) + (tid & 1);
      pair[0] = -o.hi;
      pair[2] = o.r;
      // all rows see all keys of the item: no comparisons below
      const bool all = bar_and(bar, kKeys, tid >= count || o.last >= u.end - 1);
      // a warp whose wait failed goes on to every barrier, so that none is left behind
      if (ok) {
        ok = warp_wait(&sh.s_full[grp], uint32_t(sn) & 1u, p.st, forced, abort_flag);
        if (!ok && lane == 0) *abort_flag = 1;
      }
      ++sn;
      if (!ok) return;
      tc_fence_after();
      const float unit = FP4 ? sh.unit[single ? 2 * grp + info : fills & 3][tid] : p.scale_log2;
      const float2 unit2 = make_float2(unit, unit);
      constexpr int kCols = FP4 ? 16 : 32;  // at a time; 32 would spill next to a third group's registers
      for (int c0 = 0; c0 < count; c0 += kCols) {
        uint32_t s[kCols];
        if constexpr (FP4) tmem_ld16(row + c0, s);
        else tmem_ld32(row + c0, s);
        tmem_ld_wait();
        auto pair_of_rows = [&](int j) {
          const float4 hr = sh.pair[grp][info][c0 / 2 + j];
          const float2 x = ffma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), unit2,
                                 make_float2(hr.x, hr.y));
          sum[j & 1] = ffma2(make_float2(fast_exp2(x.x), fast_exp2(x.y)), make_float2(hr.z, hr.w), sum[j & 1]);
        };
        auto one_row = [&](int j) {
          const float* hr = reinterpret_cast<const float*>(&sh.pair[grp][info][(c0 + j) >> 1]) + (j & 1);
          sum[0].x = fmaf(fast_exp2(fmaf(__uint_as_float(s[j]), unit, hr[0])), hr[2], sum[0].x);
        };
        if (all && c0 + kCols <= count) {
#pragma unroll
          for (int j = 0; j < kCols / 2; ++j) pair_of_rows(j);
        } else if (all) {
#pragma unroll
          for (int j = 0; j < kCols / 2; ++j) {
            if (c0 + 2 * j + 1 < count) pair_of_rows(j);
            else if (c0 + 2 * j < count) one_row(2 * j);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (c0 + j < count && key <= sh.last[grp][info][c0 + j]) one_row(j);
        }
      }
      tc_fence_before();
      mbar_arrive(&sh.s_empty[grp]);
    };
    auto total = [&]() { return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y); };
    const int step = single ? 2 : 1;
    int i = i0 + (single ? grp : 0);
    if (single && grp == 1 && i < i1) t = next_item(p, t);
    int page = i < i1 ? page_of(t) : 0;
    float* score = score_at(t, page);
    float old = i < i1 ? old_score(t, score) : 0.f;
    float lse = single ? lse_of(t, 0) : 0.f;
    for (; i < i1; i += step) {
      const bool more = i + step < i1;
      TileItem next = t;
      if (more) next = next_item(p, t);
      if (more && single) next = next_item(p, next);
      const int next_page = more ? page_of(next) : 0;
      float* next_score = score_at(next, next_page);
      const float next_old = more ? old_score(next, next_score) : 0.f;
      sum[0] = sum[1] = make_float2(0.f, 0.f);
      float w = 0.f;
      if (single) {
        const float next_lse = more ? lse_of(next, 0) : 0.f;
        if (t.tiles > 0) add_weights(t, t.tok0, lse);
        w = total();
        lse = next_lse;
      } else {
        for (int n = 0; n < t.tiles; ++n)
          if (((products + n) & 1) == grp) add_weights(t, t.tok0 + n * p.tile_queries, lse_of(t, n));
        products += t.tiles;
        fills += t.tiles > 0;
        w = total();
        const int par = (i - i0) & 1;
        if (grp == 1) sh.part[par][tid] = w;
        bar_and(3, 2 * kKeys, true);
        if (grp == 0) w += sh.part[par][tid];
      }
      if (t.begin + tid < t.end && ok && (single || grp == 0)) *score = is_fresh(t) ? w : fmaf(p.decay, old, w);
      t = next;
      score = next_score;
      old = next_old;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kTmem);
}

template <typename T, int D, int NT, bool FP4>
bskv_status launch_stream(const bskv_plan* plan, WeightsParams& wp, cudaStream_t st) {
  const size_t smem = size_t(kWarps) * Shape<D, FP4>::kRing;
  auto kern = weights_stream_kernel<T, D, NT, FP4>;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "attn_weights: cudaFuncSetAttribute")) return s;
  // Plans have up to 16 workers per SM. Where fewer warps fit, a warp takes two workers' chunks in a row
  // (64 requests of 512 to 4096 tokens at 8 warps per SM: 53.0 us where two waves of CTAs took 54.1).
  wp.take = wp.num_workers > int64_t(plan->num_sms) * kWarps * weights_ctas_per_sm(D, FP4) ? 2 : 1;
  const int warps = (wp.num_workers + wp.take - 1) / wp.take;
  kern<<<(warps + kWarps - 1) / kWarps, kWarps * 32, smem, st>>>(wp);
  return cuda_check(cudaGetLastError(), "attn_weights launch");
}

template <typename T, int D, bool FP4>
bskv_status launch_tile(const bskv_plan* plan, WeightsParams& wp, cudaStream_t st) {
  const int ps = plan->page_size;
  wp.box = ps % 128 == 0 ? 128 : ps % 64 == 0 ? 64 : ps % 32 == 0 ? 32 : ps % 16 == 0 ? 16 : 8;
  wp.tile_queries = std::min(kKeys / wp.group, plan->q_len);
  wp.single = plan->q_len <= wp.tile_queries;
  const CUtensorMapDataType dt = __is_same(T, __half) ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap qmap, kmap{};
  const uint64_t qd[3] = {D, uint64_t(plan->num_qo_heads), uint64_t(plan->M)};
  const uint64_t qst[2] = {uint64_t(wp.q_s1) * 2, uint64_t(wp.q_s0) * 2};
  const uint32_t qb[3] = {64, uint32_t(wp.group), uint32_t(wp.tile_queries)};
  if (bskv_status s = encode_tiled(&qmap, dt, 3, wp.q, qd, qst, qb, CU_TENSOR_MAP_SWIZZLE_128B)) return s;
  if (!FP4) {
    const uint64_t kd[5] = {D, uint64_t(ps), uint64_t(plan->num_kv_heads), 2, uint64_t(plan->num_pages)};
    const uint64_t kst[4] = {uint64_t(wp.k_s3), uint64_t(wp.k_s2), uint64_t(wp.k_s1), uint64_t(wp.k_s0)};
    const uint32_t kb[5] = {64, uint32_t(wp.box), 1, 1, 1};
    if (bskv_status s = encode_tiled(&kmap, dt, 5, wp.keys, kd, kst, kb, CU_TENSOR_MAP_SWIZZLE_128B)) return s;
  }
  const size_t smem = 1024 + size_t(3) * (D / 64) * kPanel + sizeof(TileShared);
  auto kern = weights_tile_kernel<T, D, FP4>;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "attn_weights: cudaFuncSetAttribute")) return s;
  const int per_sm = 2;  // by shared memory (96 KB for 128 dims) and TMEM (256 columns)
  wp.num_requests = meta_word(plan, H_MERGES);
  wp.num_items = meta_word(plan, H_UNITS);
  wp.queries = FastDiv(wp.tile_queries);
  const int grid = int(std::min<int64_t>(wp.num_items, int64_t(plan->num_sms) * per_sm));
  kern<<<grid, tile_threads(FP4), smem, st>>>(qmap, kmap, wp);
  return cuda_check(cudaGetLastError(), "attn_weights launch");
}

template <typename T, int D, bool FP4>
bskv_status launch(const bskv_plan* plan, WeightsParams& wp, cudaStream_t st) {
  switch (meta_word(plan, H_VARIANT)) {
    case WEIGHTS_STREAM8: return launch_stream<T, D, 1, FP4>(plan, wp, st);
    case WEIGHTS_STREAM16: return launch_stream<T, D, 2, FP4>(plan, wp, st);
    default: return launch_tile<T, D, FP4>(plan, wp, st);
  }
}

template <bool FP4>
bskv_status run(const char* who, const bskv_plan* plan, const void* q, const int64_t* q_strides,
                const float* lse, float* scores, const int64_t* scores_strides, float decay,
                float sm_scale, WeightsParams& wp, cudaStream_t st) {
  // without queries the scores fade only
  if ((plan->M > 0 && (!q || !lse)) || !q_strides || !scores || !scores_strides) { set_error("%s: NULL tensor", who); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(q) || !aligned16(scores)) { set_error("%s: tensors must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i) {
    if (q_strides[i] <= 0 || q_strides[i] % 8) { set_error("%s: q strides must be positive multiples of 8 elements", who); return BSKV_ERR_INVALID_ARG; }
  }
  for (int i = 0; i < 2; ++i) {
    if (scores_strides[i] <= 0 || scores_strides[i] % 4) {
      set_error("%s: scores stride %d (%lld) must be a positive multiple of 4 elements", who, i, (long long)scores_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  if (!(decay >= 0.f && decay <= 1.f)) { set_error("%s: decay %g outside [0, 1]", who, double(decay)); return BSKV_ERR_INVALID_ARG; }
  wp.meta = plan->meta_dev;
  wp.q = q; wp.q_s0 = q_strides[0]; wp.q_s1 = q_strides[1];
  wp.lse = lse;
  wp.scores = scores; wp.w_s0 = scores_strides[0]; wp.w_s1 = scores_strides[1];
  wp.num_kv_heads = plan->num_kv_heads;
  wp.group = plan->num_qo_heads / plan->num_kv_heads;
  wp.heads = FastDiv(plan->num_kv_heads);
  wp.groups = FastDiv(wp.group);
  wp.page_size = FastDiv(plan->page_size);
  wp.num_qo_heads = plan->num_qo_heads; wp.causal = plan->causal;
  wp.off_workers = meta_word(plan, H_OFF_WORKERS);
  wp.off_aux1 = meta_word(plan, H_OFF_AUX1);
  wp.off_req = meta_word(plan, H_OFF_MERGES);
  wp.num_workers = meta_word(plan, H_WORKERS);
  wp.off_records = plan->walk_records;
  wp.decay = decay;
  wp.scale_log2 = sm_scale_log2(sm_scale, plan->head_dim);
  if (bskv_status s = status_args(&wp.st)) return s;
  const bool bf = plan->dtype == BSKV_BF16;
  if (plan->head_dim == 128)
    return bf ? launch<__nv_bfloat16, 128, FP4>(plan, wp, st) : launch<__half, 128, FP4>(plan, wp, st);
  return bf ? launch<__nv_bfloat16, 64, FP4>(plan, wp, st) : launch<__half, 64, FP4>(plan, wp, st);
}

bskv_status check_plan(const char* who, const bskv_plan* plan) {
  if (!plan || plan->kind != KIND_WEIGHTS) { set_error("%s: not an attention-weight plan", who); return BSKV_ERR_INVALID_ARG; }
  if (!plan->meta_dev) { set_error("%s: plan not uploaded (bskv_plan_upload)", who); return BSKV_ERR_INVALID_ARG; }
  return BSKV_OK;
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_run_attn_weights(const bskv_plan* plan, const void* q,
                                             const int64_t* q_strides, const void* kv_cache,
                                             const int64_t* kv_strides, const float* lse,
                                             float* scores, const int64_t* scores_strides,
                                             float decay, float sm_scale, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_attn_weights");
  const char* who = "run_attn_weights";
  if (bskv_status s = check_plan(who, plan)) return s;
  if (meta_word(plan, H_GRID) == 0) return BSKV_OK;
  if (!kv_cache || !kv_strides || !aligned16(kv_cache)) { set_error("%s: kv_cache must be a 16-byte aligned tensor", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 4; ++i) {
    if (kv_strides[i] <= 0 || kv_strides[i] % 8) {
      set_error("%s: kv stride %d (%lld elements) must be positive and 16-byte aligned", who, i, (long long)kv_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  WeightsParams wp{};
  wp.keys = static_cast<const uint8_t*>(kv_cache);
  wp.k_s0 = 2 * kv_strides[0]; wp.k_s1 = 2 * kv_strides[1]; wp.k_s2 = 2 * kv_strides[2]; wp.k_s3 = 2 * kv_strides[3];
  return run<false>(who, plan, q, q_strides, lse, scores, scores_strides, decay, sm_scale, wp,
                    static_cast<cudaStream_t>(stream));
}

extern "C" bskv_status bskv_run_attn_weights_fp4(const bskv_plan* plan, const void* q,
                                                 const int64_t* q_strides, const void* kv_codes,
                                                 const int64_t* codes_strides,
                                                 const void* kv_scales,
                                                 const int64_t* scales_strides, const float* lse,
                                                 float* scores, const int64_t* scores_strides,
                                                 float decay, float sm_scale, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_attn_weights_fp4");
  const char* who = "run_attn_weights_fp4";
  if (bskv_status s = check_plan(who, plan)) return s;
  if (meta_word(plan, H_GRID) == 0) return BSKV_OK;
  if (bskv_status s = check_fp4_cache(who, kv_codes, codes_strides, kv_scales, scales_strides)) return s;
  WeightsParams wp{};
  wp.keys = static_cast<const uint8_t*>(kv_codes);
  wp.k_s0 = codes_strides[0]; wp.k_s1 = codes_strides[1]; wp.k_s2 = codes_strides[2]; wp.k_s3 = codes_strides[3];
  wp.scales = static_cast<const uint8_t*>(kv_scales);
  wp.s_s0 = scales_strides[0]; wp.s_s2 = scales_strides[2];
  return run<true>(who, plan, q, q_strides, lse, scores, scores_strides, decay, sm_scale, wp,
                   static_cast<cudaStream_t>(stream));
}
