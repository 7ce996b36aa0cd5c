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
// Keys are the M = 16 rows of mma.sync m16n8k16, query rows (token, head) its N = 8 columns, so a
// key's sum stays in its lanes until one reduction over the four lanes of its row. A row's lane
// reads 16-byte chunks t, t + 4, ...: products of chunk c with the same chunk of the query are
// two k-steps, whatever the order of the dims. Two kernels:
//   * stream (up to 16 query rows a request, the decode step): query fragments stay in
//     registers, each warp streams a range of tokens through a private ring of 32-token tiles
//     filled by 16-byte asynchronous copies; bound by reading K (HBM).
//   * tile (more rows, a prefill window): a CTA keeps the fragments of 128 keys in registers and
//     passes the query rows, staged in shared memory 64 at a time, over them; a warp's 32 keys
//     halve the shared-memory reads per product against 16. Bound by the tensor pipe and exp.
// 4-bit keys (E2M1 codes times 2^x per 32 values): the stream kernel multiplies codes and f16
// queries and scales each block's fp32 partial sum; the tile kernel turns a key once into the
// query's type, relative to its largest scale, and multiplies that back after the product.
#include <math.h>

#include <type_traits>

#include "common.cuh"
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
constexpr int kKeys = kWeightsKeys;  // keys per CTA of the tile kernel
constexpr int kRows = 64;            // query rows staged at a time

struct WeightsParams {
  const int32_t* meta;
  const void* q;
  int64_t q_s0, q_s1;
  const uint8_t* keys;              // 16-bit keys or codes
  int64_t k_s0, k_s2, k_s3;         // bytes: page, kv head, slot
  const uint8_t* scales;            // 4-bit keys
  int64_t s_s0, s_s2;               // bytes
  const float* lse;
  float* scores;
  int64_t w_s0, w_s1;               // floats: page, kv head
  int num_kv_heads, group, page_size, num_qo_heads, causal;
  int off_workers, off_chunks, off_records, off_aux0, off_aux1, off_req, num_workers;
  float decay, scale_log2;
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
__device__ __forceinline__ RowInfo row_info(const WeightsParams& p, const Request& rq, int kvh, int row) {
  RowInfo o{0.f, 0.f, -1};
  const int t = row / p.group;
  if (t >= rq.nq) return o;
  const float lse = __ldg(p.lse + int64_t(rq.qo + t) * p.num_qo_heads + kvh * p.group + (row - t * p.group));
  if (lse == -INFINITY) return o;
  constexpr float kLog2eLow = 1.925963033500011e-8f;  // log2 e - fp32(log2 e)
  o.hi = lse * kLog2e;
  const float lo = isinf(o.hi) ? 0.f : fmaf(lse, kLog2e, -o.hi) + lse * kLog2eLow;
  o.r = exp2f(-lo);
  o.last = p.causal ? t + rq.len - rq.nq : INT32_MAX;
  return o;
}

__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
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
  static constexpr int kRing = kStages * ((kStage + 15) / 16 * 16);
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
    const int row = 8 * nt + g, tok = row / p.group;
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
      s.info[2 * nt + e] = row_info(p, rq, kvh, 8 * nt + 2 * t + e);
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
  const int w = blockIdx.x * kWarps + warp;
  if (w >= p.num_workers) return;
  const int c0 = __ldg(p.meta + p.off_workers + w), nck = __ldg(p.meta + p.off_workers + w + 1) - c0;
  const int32_t* records = p.meta + p.off_records + c0 * kWalkWords;
  PageWalk walk(records, nck, p.meta + p.off_aux1, p.num_kv_heads, p.page_size, lane);
  const bool old = p.decay != 0.f;

  constexpr int kStep = 32 / Sh::kParts;  // rows one copy instruction of the warp covers
  const int row_in = lane / Sh::kParts, part = lane % Sh::kParts;
  constexpr int kPer = FP4 ? 16 / Sh::kBlocks : 8, kCopies = kTile / kPer;  // tokens per 16 bytes of scales
  const int s_row = lane % kCopies * kPer, w_row = (lane & 7) * 4;
  int64_t k_off = 0, s_off = 0, w_off = 0;
  auto issue = [&](int stage) {
    if (walk.live()) {
      if (walk.enter()) {
        k_off = walk.page * p.k_s0 + walk.kvh * p.k_s2 + walk.slot * p.k_s3;
        if constexpr (FP4) s_off = walk.page * p.s_s0 + walk.kvh * p.s_s2 + walk.slot * Sh::kBlocks;
        w_off = walk.page * p.w_s0 + walk.kvh * p.w_s1 + walk.slot;
      }
      uint8_t* st = ring + stage * kStride;
      auto copy = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < kTile / kStep; ++i) {
          const int r = row_in + i * kStep;
          const int64_t off = walk.of_group(k_off, r);
          if (whole || walk.has(r))
            cp_async_16(st + r * Sh::kRow + (Sh::part(r, part) << 4), p.keys + off + (r & 7) * p.k_s3 + part * 16);
        }
        if constexpr (FP4) {
          const int64_t off = walk.of_group(s_off, s_row);
          if ((whole || walk.has(s_row)) && lane < kCopies)
            cp_async_16(st + Sh::kScales + 16 * lane, p.scales + off + (s_row & 7) * Sh::kBlocks);
        }
        const int64_t off = walk.of_group(w_off, w_row);  // four scores
        if ((whole || walk.has(w_row)) && lane < 8) {
          if (old) cp_async_16(st + Sh::kOld + 16 * lane, p.scores + off + (w_row & 7));
          if ((lane & 1) == 0) *reinterpret_cast<int64_t*>(st + Sh::kPlace + 4 * lane) = off;
        }
      };
      if (walk.tok + kTile <= walk.end) copy(std::true_type{});
      else copy(std::false_type{});
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
    const int b = ch.unit / p.num_kv_heads, kvh = ch.unit - b * p.num_kv_heads;
    const Request rq = request_of(p, b);
    load_rows<T, D, NT, FP4>(p, rq, kvh, lane, s);
    for (int at = ch.begin; at < ch.end; at += kTile, ++done) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // the tile is there for every lane, and the stage refilled next is free
      issue((done + kStages - 1) % kStages);
      const uint8_t* st = ring + (done % kStages) * kStride;
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
            if (key <= s.info[j].last) a = fmaf(e, s.info[j].r, a);
          }
          sum[2 * h + i] = quad_sum(a);
        }
      }
      // lane (g, t) writes key at + 8 t + g
      const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
      const int r = 8 * t + g;
      if (at + r < ch.end) {
        float* dst = p.scores + *reinterpret_cast<const int64_t*>(st + Sh::kPlace + 8 * t) + g;
        const bool fresh = !old || at + r >= rq.len - rq.nq;
        *dst = fresh ? mine : fmaf(p.decay, *reinterpret_cast<const float*>(st + Sh::kOld + 4 * r), mine);
      }
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------------------
// tile kernel
// ---------------------------------------------------------------------------------------

// 16 bytes (8 values) of a 4-bit key as a fragment chunk of T, in units of the row's largest scale.
template <typename T>
__device__ __forceinline__ uint4 widen(uint32_t w, float f) {
  uint32_t h[4], o[4];
  cvt_e2m1x8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    o[i] = MmaOp<T>::pack(a.x * f, a.y * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D, bool FP4>
__global__ void __launch_bounds__(kKeys) weights_tile_kernel(const WeightsParams p) {
  constexpr int kRowBytes = 2 * D, kParts = kRowBytes / 16, kThreads = kKeys;
  __shared__ __align__(128) uint8_t qs[2][kRows * kRowBytes];
  __shared__ float2 row_hi_r[2][kRows];
  __shared__ int row_last[2][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kvh = blockIdx.y;
  const int4 ch = __ldg(reinterpret_cast<const int4*>(p.meta + p.off_chunks) + blockIdx.x);
  const int b = ch.x;  // {request, first key, end key, 0}
  const Request rq = request_of(p, b);
  const int pbase = __ldg(p.meta + p.off_aux0 + b);
  const int32_t* pages = p.meta + p.off_aux1 + pbase;
  const int nrows = rq.nq * p.group;
  // causal: the first query that sees the tile's first key
  const int row0 = p.causal ? max(0, ch.y - (rq.len - rq.nq)) * p.group : 0;

  auto stage = [&](int buf, int first) {
    for (int c = threadIdx.x; c < kRows * kParts; c += kThreads) {
      const int r = c / kParts, part = c % kParts, row = first + r;
      uint8_t* dst = qs[buf] + r * kRowBytes + ((part ^ ((r & 1) << 2)) << 4);
      if (row < nrows) {
        const int tok = row / p.group;
        cp_async_16(dst, static_cast<const T*>(p.q) + int64_t(rq.qo + tok) * p.q_s0 +
                             (int64_t(kvh) * p.group + (row - tok * p.group)) * p.q_s1 + part * 8);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
    }
    cp_async_commit();
    if (threadIdx.x < kRows) {
      const RowInfo o = row_info(p, rq, kvh, first + threadIdx.x);
      row_hi_r[buf][threadIdx.x] = make_float2(o.hi, o.r);
      row_last[buf][threadIdx.x] = o.last;
    }
  };
  if (row0 < nrows) stage(0, row0);

  // this warp's 32 keys as A fragments, straight from the cache; row i of a lane is key
  // ch.y + 32 warp + 8 i + g
  uint4 a[D / 32][4];
  float unit[4];
  const int key0 = ch.y + 32 * warp;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key0 + 8 * i + g;
    unit[i] = p.scale_log2;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) a[j][i] = make_uint4(0, 0, 0, 0);
    if (key < ch.z) {
      const int n = key / p.page_size, sl = key - n * p.page_size;
      const int64_t pg = __ldg(pages + n);
      const uint8_t* src = p.keys + pg * p.k_s0 + kvh * p.k_s2 + sl * p.k_s3;
      if constexpr (FP4) {
        const uint8_t* sc = p.scales + pg * p.s_s0 + kvh * p.s_s2;
        uint32_t code[D / 32], top = 0;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          code[j] = __ldg(sc + sl * (D / 32) + j);
          bad = bad || code[j] == 255u;
          top = max(top, code[j]);
        }
        unit[i] = bad ? NAN : p.scale_log2 * e8m0_value(top);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          a[j][i] = widen<T>(__ldg(reinterpret_cast<const uint32_t*>(src + 16 * j + 4 * t)),
                             top - code[j] > 126u ? 0.f : pow2(int(code[j]) - int(top)));
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) a[j][i] = __ldg(reinterpret_cast<const uint4*>(src + 64 * j + 16 * t));
      }
    }
  }

  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int buf = 0;
  for (int first = row0; first < nrows; first += kRows, buf ^= 1) {
    cp_async_wait<0>();
    __syncthreads();  // this block of rows is there, and everyone is done with the other buffer
    if (first + kRows < nrows) stage(buf ^ 1, first + kRows);
    const int tiles = (min(kRows, nrows - first) + 7) / 8;
    for (int n = 0; n < tiles; ++n) {
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const uint8_t* qr = qs[buf] + (8 * n + g) * kRowBytes;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(qr + (((t + 4 * j) ^ ((g & 1) << 2)) << 4));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 &u = a[j][2 * m], &v = a[j][2 * m + 1];
          const uint32_t f0[4] = {u.x, v.x, u.y, v.y}, f1[4] = {u.z, v.z, u.w, v.w};
          MmaOp<T>::run(acc[m], f0, x.x, x.y);
          MmaOp<T>::run(acc[m], f1, x.z, x.w);
        }
      }
      const float4 hr = *reinterpret_cast<const float4*>(&row_hi_r[buf][8 * n + 2 * t]);
      const int2 last = *reinterpret_cast<const int2*>(&row_last[buf][8 * n + 2 * t]);
      const bool all = __all_sync(0xffffffffu, min(last.x, last.y) >= key0 + 31);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e0 = fast_exp2(fmaf(acc[i >> 1][2 * (i & 1)], unit[i], -hr.x));
        const float e1 = fast_exp2(fmaf(acc[i >> 1][2 * (i & 1) + 1], unit[i], -hr.z));
        const int key = key0 + 8 * i + g;
        if (all || key <= last.x) sum[i] = fmaf(e0, hr.y, sum[i]);
        if (all || key <= last.y) sum[i] = fmaf(e1, hr.w, sum[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = quad_sum(sum[i]);
  const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
  const int key = key0 + 8 * t + g;
  if (key < ch.z) {
    const int n = key / p.page_size, sl = key - n * p.page_size;
    float* dst = p.scores + __ldg(pages + n) * p.w_s0 + kvh * p.w_s1 + sl;
    const bool fresh = p.decay == 0.f || key >= rq.len - rq.nq;
    *dst = fresh ? mine : fmaf(p.decay, *dst, mine);
  }
}

template <typename T, int D, int NT, bool FP4>
bskv_status launch_stream(const bskv_plan* plan, const WeightsParams& wp, cudaStream_t st) {
  const size_t smem = size_t(kWarps) * Shape<D, FP4>::kRing;
  auto kern = weights_stream_kernel<T, D, NT, FP4>;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "attn_weights: cudaFuncSetAttribute")) return s;
  kern<<<meta_word(plan, H_GRID), kWarps * 32, smem, st>>>(wp);
  return cuda_check(cudaGetLastError(), "attn_weights launch");
}

template <typename T, int D, bool FP4>
bskv_status launch(const bskv_plan* plan, const WeightsParams& wp, cudaStream_t st) {
  switch (meta_word(plan, H_VARIANT)) {
    case WEIGHTS_STREAM8: return launch_stream<T, D, 1, FP4>(plan, wp, st);
    case WEIGHTS_STREAM16: return launch_stream<T, D, 2, FP4>(plan, wp, st);
    default: break;
  }
  weights_tile_kernel<T, D, FP4><<<dim3(unsigned(meta_word(plan, H_GRID)), unsigned(wp.num_kv_heads)), kKeys, 0, st>>>(wp);
  return cuda_check(cudaGetLastError(), "attn_weights launch");
}

template <bool FP4>
bskv_status run(const char* who, const bskv_plan* plan, const void* q, const int64_t* q_strides,
                const float* lse, float* scores, const int64_t* scores_strides, float decay,
                float sm_scale, WeightsParams& wp, cudaStream_t st) {
  if (!q || !q_strides || !lse || !scores || !scores_strides) { set_error("%s: NULL tensor", who); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(q) || !aligned16(scores)) { set_error("%s: tensors must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  if (q_strides[0] % 8 || q_strides[1] % 8) { set_error("%s: q strides must be multiples of 8 elements", who); return BSKV_ERR_INVALID_ARG; }
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
  wp.page_size = plan->page_size; wp.num_qo_heads = plan->num_qo_heads; wp.causal = plan->causal;
  wp.off_workers = meta_word(plan, H_OFF_WORKERS);
  wp.off_chunks = meta_word(plan, H_OFF_CHUNKS);
  wp.off_aux0 = meta_word(plan, H_OFF_AUX0);
  wp.off_aux1 = meta_word(plan, H_OFF_AUX1);
  wp.off_req = meta_word(plan, H_OFF_MERGES);
  wp.num_workers = meta_word(plan, H_WORKERS);
  wp.off_records = plan->walk_records;
  wp.decay = decay;
  wp.scale_log2 = sm_scale_log2(sm_scale, plan->head_dim);
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
  wp.k_s0 = 2 * kv_strides[0]; wp.k_s2 = 2 * kv_strides[2]; wp.k_s3 = 2 * kv_strides[3];
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
  wp.k_s0 = codes_strides[0]; wp.k_s2 = codes_strides[2]; wp.k_s3 = codes_strides[3];
  wp.scales = static_cast<const uint8_t*>(kv_scales);
  wp.s_s0 = scales_strides[0]; wp.s_s2 = scales_strides[2];
  return run<true>(who, plan, q, q_strides, lse, scores, scores_strides, decay, sm_scale, wp,
                   static_cast<cudaStream_t>(stream));
}
