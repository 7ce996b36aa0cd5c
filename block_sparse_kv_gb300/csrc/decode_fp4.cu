// Paged-KV batch decode over a microscaled 4-bit cache, with split-KV and the LSE merge.
//
// Mathematics. K[j, d] = e_K[j, d] X[j, d / 32] with E2M1 codes e and power-of-two scales X
// (and V alike), so
//   q.k_j  = sum_blocks X_K[j, b] (sum_{d in b} q_d e_K[j, d])
//   o_d    = sum_j (p_j X_V[j, d / 32]) e_V[j, d]
// The codes are exact in f16, so both inner sums are f16 tensor-core products of the codes
// themselves: a key's scale multiplies the fp32 partial sum of its block, a value's scale is
// folded into the softmax weight. Queries in bf16 are made f16 by an exact power of two per
// head. The weight times scale is rounded to f16 (half a step, 2^-11 relative) relative to a
// power of two per (head, block) that follows the largest product so far, so the scales may
// have any magnitude: rr below.
//
// Tokens are the M = 16 rows of mma.sync m16n8k16 and the query heads of a kv head its N = 8
// columns (two column tiles above 8 heads): with heads as rows a group of 4 would leave three
// quarters of each product unused. S^T = K Q^T, O^T = V^T P^T; P^T reaches its operand layout
// by movmatrix. Layouts that the fragments need come from which lane reads which word:
//   * K: lane (g, t) reads word t of each 16-byte block of tokens g and g + 8; its 8 values are
//     two k-steps, the query fragment is loaded in the same order.
//   * V: lane (g, t) reads the 4 values 32 b + 4 g .. + 3 of tokens 2t, 2t + 1, 2t + 8, 2t + 9;
//     two logic operations pair the nibbles of two tokens in a byte, and
//     cvt.rn.f16x2.e2m1x2 then yields the (token, token + 1) pairs of the A operand.
//
// What bounds it: the cache is read once, 136 bytes per token and kv head of 128 dims against
// 512 in 16 bits, so instructions issued per byte are what to save; see the measured figures at
// kFp4WarpsPerSm. Each warp is a worker of its own over a range of one or more (request, kv
// head) units, with a private ring of 32-token tiles filled by 16-byte asynchronous copies
// (any page size and stride, no swizzle constraint on the page layout). A unit cut between
// workers is merged in the same launch as in the 16-bit decode, by the same code.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.h"
#include "page_walk.cuh"
#include "split_merge.cuh"

namespace bskv {
namespace {

using namespace dev;

constexpr int kTile = kFp4Tile;  // tokens per stage
static_assert(kTile == kWalkTile, "one walk step per stage");
constexpr int kWarps = kFp4Warps;
constexpr int kStages = 3;

struct Fp4DecodeParams {
  const int32_t* meta;
  const void* q;
  int64_t q_s0, q_s1;
  const uint8_t* codes;
  int64_t c_s0, c_s1, c_s2, c_s3;  // bytes
  const uint8_t* scales;
  int64_t s_s0, s_s1, s_s2;  // bytes
  void* out;
  int64_t o_s0, o_s1;
  float* lse;
  float* ws_o;
  float* ws_lse;
  int* counters;  // non-null: the last worker to finish a split unit merges it
  int num_kv_heads, group, page_size, num_qo_heads;
  int off_workers, off_chunks, off_merges, off_aux0, off_aux1, num_merges, num_workers;
  float scale_log2;
};

template <int D>
struct Shape {
  static constexpr int kBlocks = D / kFp4Block;           // scales per row
  static constexpr int kRow = D / 2;                      // bytes of codes per row
  static constexpr int kParts = kRow / 16;                // 16-byte parts per row
  static constexpr int kV = kTile * kRow;                 // stage offsets
  static constexpr int kKs = 2 * kTile * kRow;
  static constexpr int kVs = kKs + kTile * kBlocks;
  static constexpr int kStage = kKs + 2 * kTile * kBlocks;
  // Part c of row r is stored at part c ^ (r / (8 / kParts) mod kParts): the word and
  // half-word reads of the compute loop then fall into distinct banks.
  static constexpr int kSwzShift = D == 128 ? 1 : 2;
};

// Transpose of an 8x8 matrix of 16-bit elements spread over the warp as mma fragments.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Everything a warp keeps of the unit it works on. Column j of a lane is query head
// 8 (j / 2) + 2 t + (j & 1) of the kv head's group.
template <int D, int NT>
struct State {
  uint32_t q[NT][Shape<D>::kBlocks][4];     // query fragments (B operand), f16
  float o[NT][Shape<D>::kBlocks][2][4];     // O^T accumulators, in units of 1 / rr
  float m[2 * NT], l[2 * NT], c[2 * NT];    // maximum of q.k, sum, logit scale (base 2, > 0)
  float rr[2 * NT][Shape<D>::kBlocks];      // power of two that p * scale is multiplied by
};

template <typename T, int D, int NT>
__device__ __forceinline__ void load_q(const Fp4DecodeParams& p, int b, int kvh, int lane,
                                       State<D, NT>& s) {
  constexpr int NB = Shape<D>::kBlocks;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = 8 * nt + g;
    const float back = load_q_f16<T, NB>(
        static_cast<const T*>(p.q) + b * p.q_s0 + (int64_t(kvh) * p.group + h) * p.q_s1,
        h < p.group, p.scale_log2 < 0.f, lane, s.q[nt]);
    // columns 2t and 2t + 1 belong to the heads of lanes 8t and 8t + 4
    s.c[2 * nt] = fabsf(p.scale_log2) * __shfl_sync(0xffffffffu, back, 8 * t);
    s.c[2 * nt + 1] = fabsf(p.scale_log2) * __shfl_sync(0xffffffffu, back, 8 * t + 4);
  }
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    s.m[j] = -INFINITY;
    s.l[j] = 0.f;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) s.rr[j][blk] = pow2(127);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 8; ++i) s.o[nt][blk][i >> 2][i & 3] = 0.f;
}

// Multiply the accumulators of column j, block blk by f (column j is elements j & 1 and
// (j & 1) + 2 of its tile's fragments).
template <int D, int NT>
__device__ __forceinline__ void scale_o(State<D, NT>& s, int j, int blk, float f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s.o[j >> 1][blk][i][j & 1] *= f;
    s.o[j >> 1][blk][i][(j & 1) + 2] *= f;
  }
}

// One 32-token tile in shared memory; with WHOLE false, tokens >= valid lie past the chunk.
template <int D, int NT, bool WHOLE>
__device__ __forceinline__ void tile(const uint8_t* st, int valid, int lane, State<D, NT>& s) {
  using Sh = Shape<D>;
  using Mma = MmaOp<__half>;
  constexpr int NB = Sh::kBlocks;
  const int g = lane >> 2, t = lane & 3;
  const int kx = (g >> Sh::kSwzShift) & (Sh::kParts - 1);
  const int vx = ((2 * t) >> Sh::kSwzShift) & (Sh::kParts - 1);
  float x[2][NT][4];  // q.k, then weights: [16-token half][column tile][fragment]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r0 = 16 * h + g, r1 = r0 + 8;
    float s0[NB], s1[NB];
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r0), s0);
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r1), s1);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint8_t* at = st + ((blk ^ kx) << 4) + 4 * t;
      uint32_t a0[4], a1[4];
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at + r0 * Sh::kRow), a0);
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at + r1 * Sh::kRow), a1);
      const uint32_t f0[4] = {a0[0], a1[0], a0[1], a1[1]}, f1[4] = {a0[2], a1[2], a0[3], a1[3]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        Mma::run(acc, f0, s.q[nt][blk][0], s.q[nt][blk][1]);
        Mma::run(acc, f1, s.q[nt][blk][2], s.q[nt][blk][3]);
        x[h][nt][0] = blk ? fmaf(acc[0], s0[blk], x[h][nt][0]) : acc[0] * s0[blk];
        x[h][nt][1] = blk ? fmaf(acc[1], s0[blk], x[h][nt][1]) : acc[1] * s0[blk];
        x[h][nt][2] = blk ? fmaf(acc[2], s1[blk], x[h][nt][2]) : acc[2] * s1[blk];
        x[h][nt][3] = blk ? fmaf(acc[3], s1[blk], x[h][nt][3]) : acc[3] * s1[blk];
      }
    }
    if constexpr (!WHOLE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * h + 8 * (i >> 1) + g >= valid) x[h][nt][i] = -INFINITY;
    }
  }
  // online softmax, column by column
  float mn[2 * NT];
  bool up = false;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int e = j & 1;
    mn[j] = fmaxf(fmaxf(x[0][j >> 1][e], x[0][j >> 1][e + 2]), fmaxf(x[1][j >> 1][e], x[1][j >> 1][e + 2]));
    mn[j] = fmaxf(s.m[j], max_over_rows(mn[j]));
    up = up || mn[j] > s.m[j];
  }
  if (__any_sync(0xffffffffu, up)) {
    // A higher maximum: weights so far shrink by 2^-(mn - m). rr grows by the next whole
    // power of two, so that p * scale * rr of a given product never becomes smaller.
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const float delta = (mn[j] - s.m[j]) * s.c[j];
      const float alpha = fast_exp2(-delta);
      s.l[j] *= alpha;
      const int grow = int(fminf(ceilf(delta), 254.f));
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        const int k = exponent_of(s.rr[j][blk]);
        const int kn = min(k + grow, 127);
        scale_o(s, j, blk, fast_exp2(float(kn - k) - delta));
        s.rr[j][blk] = pow2(kn);
      }
      s.m[j] = mn[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const float mc = s.m[j] * s.c[j];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float& v = x[h][j >> 1][(j & 1) + 2 * i];
        v = fast_exp2(fmaf(v, s.c[j], -mc));
        s.l[j] += v;
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // weights times value scales, as f16 pairs of two heads
    float f[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * h + 8 * i + g;
      uint32_t w = scale_word<D>(st + Sh::kVs, r);
      if constexpr (!WHOLE) w = r < valid ? w : 0u;
      scales_of<NB>(w, f[i]);
    }
    uint32_t pp[NT][NB][2];
    for (int round = 0; round < 2; ++round) {
      __half2 top = __float2half2_rn(0.f);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t w = pack_half2(x[h][nt][2 * i] * s.rr[2 * nt][blk] * f[i][blk],
                                          x[h][nt][2 * i + 1] * s.rr[2 * nt + 1][blk] * f[i][blk]);
            pp[nt][blk][i] = w;
            top = __hmax2(top, *reinterpret_cast<const __half2*>(&w));
          }
        }
      // up to 2^15 the products are safe in f16; above, lower rr so that the largest becomes
      // [2^10, 2^11): products 2^-24 of it still keep 11 bits, and smaller ones are off by at
      // most 2^-35 of it
      const bool over = __hgt(__hmax(__low2half(top), __high2half(top)), __float2half(32768.f));
      if (round == 1 || !__any_sync(0xffffffffu, over)) break;
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j)
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          float big = fmaxf(x[h][j >> 1][j & 1] * f[0][blk],
                            x[h][j >> 1][(j & 1) + 2] * f[1][blk]);
          big = max_over_rows(big);
          const int k = exponent_of(s.rr[j][blk]);
          const int kn = min(k, max(-126, 10 - exponent_of(big)));
          scale_o(s, j, blk, fast_exp2(float(kn - k)));
          s.rr[j][blk] = pow2(kn);
        }
    }
    // O^T += V^T P^T
    const uint8_t* row = st + Sh::kV + (16 * h + 2 * t) * Sh::kRow + 2 * g;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint8_t* at = row + ((blk ^ vx) << 4);
      const uint32_t h0 = *reinterpret_cast<const uint16_t*>(at);
      const uint32_t h1 = *reinterpret_cast<const uint16_t*>(at + Sh::kRow);
      const uint32_t h2 = *reinterpret_cast<const uint16_t*>(at + 8 * Sh::kRow);
      const uint32_t h3 = *reinterpret_cast<const uint16_t*>(at + 9 * Sh::kRow);
      uint32_t a[2][4];  // rows g / g + 8 of the two products: values 4g + {0, 1} and {2, 3}
      cvt_e2m1x4((h0 & 0x0f0fu) | ((h1 << 4) & 0xf0f0u), a[0][0], a[1][0]);
      cvt_e2m1x4(((h0 >> 4) & 0x0f0fu) | (h1 & 0xf0f0u), a[0][1], a[1][1]);
      cvt_e2m1x4((h2 & 0x0f0fu) | ((h3 << 4) & 0xf0f0u), a[0][2], a[1][2]);
      cvt_e2m1x4(((h2 >> 4) & 0x0f0fu) | (h3 & 0xf0f0u), a[0][3], a[1][3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t b0 = movmatrix(pp[nt][blk][0]), b1 = movmatrix(pp[nt][blk][1]);
        Mma::run(s.o[nt][blk][0], a[0], b0, b1);
        Mma::run(s.o[nt][blk][1], a[1], b0, b1);
      }
    }
  }
}

// Normalise a finished chunk and write it to out / lse (slot < 0) or as a partial state.
template <typename T, int D, int NT>
__device__ __forceinline__ void finish(const Fp4DecodeParams& p, int b, int kvh, int slot, int lane,
                                       State<D, NT>& s) {
  using Mma = MmaOp<T>;
  constexpr int NB = Shape<D>::kBlocks;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int h = 8 * (j >> 1) + 2 * t + (j & 1);
    const float l = sum_over_rows(s.l[j]);
    const float inv = 1.f / l, lse = fmaf(s.m[j], s.c[j], __log2f(l)) * kLn2;
    if (h >= p.group) continue;
    if (g == 0) {
      if (slot >= 0) p.ws_lse[int64_t(slot) * p.group + h] = lse;
      else if (p.lse) p.lse[int64_t(b) * p.num_qo_heads + kvh * p.group + h] = lse;
    }
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const float f = pow2_inverse(s.rr[j][blk]) * inv;
      const auto& o = s.o[j >> 1][blk];
      const int e = j & 1;
      const float4 v = make_float4(o[0][e] * f, o[0][e + 2] * f, o[1][e] * f, o[1][e + 2] * f);
      const int d = 32 * blk + 4 * g;
      if (slot >= 0) {
        *reinterpret_cast<float4*>(p.ws_o + (int64_t(slot) * p.group + h) * D + d) = v;
      } else {
        T* dst = static_cast<T*>(p.out) + b * p.o_s0 + (int64_t(kvh) * p.group + h) * p.o_s1 + d;
        *reinterpret_cast<uint2*>(dst) = make_uint2(Mma::pack(v.x, v.y), Mma::pack(v.z, v.w));
      }
    }
  }
}

template <typename T, int D>
__device__ __noinline__ void merge_unit(const Fp4DecodeParams& p, int lane, int unit, int first,
                                        int count) {
  const int b = unit / p.num_kv_heads, h = unit % p.num_kv_heads * p.group;
  merge_rows<T, D, 4, 2>(lane, p.ws_o, p.ws_lse, first, count, p.group, 0, p.group,
                         static_cast<T*>(p.out) + b * p.o_s0 + int64_t(h) * p.o_s1, p.o_s1,
                         p.lse ? p.lse + int64_t(b) * p.num_qo_heads + h : nullptr);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, fp4_ctas_per_sm(NT))
    decode_fp4_kernel(const Fp4DecodeParams p) {
  using Sh = Shape<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * (kStages * Sh::kStage);
  const int P = p.num_workers;
  const int w = blockIdx.x * kWarps + warp;
  if (w >= P) return;
  const int32_t* merges = p.meta + p.off_merges;
  const int Hkv = p.num_kv_heads;
  PageWalk walk(p.meta, p.off_workers, p.off_chunks, p.off_aux0, p.off_aux1, w, Hkv, p.page_size, lane);
  const int nck = walk.count();

  // Part of a row that this lane copies, and the 16 bytes of scales: their place relative to the
  // row's group of 8 tokens, whose own offsets the group's lane keeps.
  const int row_in = lane / Sh::kParts, part = lane % Sh::kParts;
  const uint8_t* k_lane = p.codes + (row_in & 7) * p.c_s3 + part * 16;
  const uint8_t* v_lane = k_lane + p.c_s1;
  constexpr int kPer = 16 / Sh::kBlocks;  // tokens per 16 bytes of scales
  constexpr int kCopies = kTile / kPer;
  const int s_row = lane % kCopies * kPer, which = (lane / kCopies) & 1;
  const uint8_t* s_lane = p.scales + which * p.s_s1 + (s_row & 7) * Sh::kBlocks;
  uint8_t* to_lane = ring + row_in * Sh::kRow + ((part ^ ((row_in >> Sh::kSwzShift) & (Sh::kParts - 1))) << 4);
  uint8_t* s_to_lane = ring + Sh::kKs + which * kTile * Sh::kBlocks + lane % kCopies * 16;
  int64_t c_off = 0, s_off = 0;
  auto issue = [&](int stage) {
    if (walk.live()) {
      if (walk.enter()) {
        c_off = walk.page * p.c_s0 + walk.kvh * p.c_s2 + walk.slot * p.c_s3;
        s_off = walk.page * p.s_s0 + walk.kvh * p.s_s2 + walk.slot * Sh::kBlocks;
      }
      auto copy = [&](auto whole) {
        uint8_t* to = to_lane + stage * Sh::kStage;
#pragma unroll
        for (int i = 0; i < Sh::kParts; ++i) {
          const int r = row_in + i * (32 / Sh::kParts);
          const int64_t off = walk.of_group(c_off, r);
          if (whole || walk.has(r)) {
            cp_async_16(to + i * (32 / Sh::kParts) * Sh::kRow, k_lane + off);
            cp_async_16(to + i * (32 / Sh::kParts) * Sh::kRow + Sh::kV, v_lane + off);
          }
        }
        const int64_t off = walk.of_group(s_off, s_row);
        if ((whole || walk.has(s_row)) && lane < 2 * kCopies)
          cp_async_16(s_to_lane + stage * Sh::kStage, s_lane + off);
      };
      if (walk.tok + kTile <= walk.end) copy(std::true_type{});
      else copy(std::false_type{});
      walk.advance();
    }
    cp_async_commit();
  };

  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // Units without tokens are zero-filled by the workers in turn.
  if (p.counters)
    for (int i = w; i < p.num_merges; i += P)
      if (merges[3 * i + 2] == 0) merge_unit<T, D>(p, lane, merges[3 * i], 0, 0);

  State<D, NT> s;
  int done = 0;
  for (int k = 0; k < nck; ++k) {
    const int4 ch = walk.chunk(k);
    const int b = ch.x / Hkv, kvh = ch.x - b * Hkv;
    load_q<T, D, NT>(p, b, kvh, lane, s);
    for (int at = ch.y; at < ch.z; at += kTile, ++done) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // the tile is there for every lane, and the stage refilled next is free
      issue((done + kStages - 1) % kStages);
      const uint8_t* st = ring + (done % kStages) * Sh::kStage;
      if (ch.z - at >= kTile) tile<D, NT, true>(st, kTile, lane, s);
      else tile<D, NT, false>(st, ch.z - at, lane, s);
    }
    finish<T, D, NT>(p, b, kvh, ch.w, lane, s);
    if (ch.w >= 0 && p.counters) {
      // The last of the unit's chunks to finish merges all of them (release / acquire through
      // lane 0's atomic, the other lanes' writes ordered before it by the __syncwarp).
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        const int item = find_merge_item(merges, p.num_merges, ch.x);
        last = atomic_add_acq_rel(p.counters + item, 1) == merges[3 * item + 2] - 1 ? item + 1 : 0;
      }
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) {
        merge_unit<T, D>(p, lane, ch.x, merges[3 * (last - 1) + 1], merges[3 * (last - 1) + 2]);
        if (lane == 0) p.counters[last - 1] = 0;  // ready for the next run
      }
    }
  }
  cp_async_wait<0>();
}

template <typename T, int D, int NT>
bskv_status launch(const bskv_plan* plan, const Fp4DecodeParams& dp, cudaStream_t st) {
  const size_t smem = size_t(kWarps) * kStages * Shape<D>::kStage;
  auto kern = decode_fp4_kernel<T, D, NT>;
  if (bskv_status s = cuda_check(
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)),
          "decode_fp4: cudaFuncSetAttribute"))
    return s;
  kern<<<meta_word(plan, H_GRID), kWarps * 32, smem, st>>>(dp);
  return cuda_check(cudaGetLastError(), "decode_fp4 kernel launch");
}

template <typename T>
bskv_status launch_t(const bskv_plan* plan, const Fp4DecodeParams& dp, cudaStream_t st) {
  const bool wide = dp.group > 8;
  if (plan->head_dim == 128) return wide ? launch<T, 128, 2>(plan, dp, st) : launch<T, 128, 1>(plan, dp, st);
  return wide ? launch<T, 64, 2>(plan, dp, st) : launch<T, 64, 1>(plan, dp, st);
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_run_decode_fp4(const bskv_plan* plan, const void* q,
                                           const int64_t* q_strides, const void* kv_codes,
                                           const int64_t* codes_strides, const void* kv_scales,
                                           const int64_t* scales_strides, void* out,
                                           const int64_t* out_strides, float* lse, float sm_scale,
                                           void* float_ws, size_t float_ws_bytes, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_decode_fp4");
  if (!plan || plan->kind != KIND_DECODE_FP4) { set_error("run_decode_fp4: not a 4-bit decode plan"); return BSKV_ERR_INVALID_ARG; }
  if (!plan->meta_dev) { set_error("run_decode_fp4: plan not uploaded (bskv_plan_upload)"); return BSKV_ERR_INVALID_ARG; }
  if (float_ws_bytes < plan->float_ws_bytes || (plan->float_ws_bytes && !float_ws)) {
    set_error("run_decode_fp4: float workspace of %zu bytes, %zu needed", float_ws_bytes, plan->float_ws_bytes);
    return BSKV_ERR_WORKSPACE_TOO_SMALL;
  }
  if (plan->batch == 0) return BSKV_OK;
  if (!q || !out || !q_strides || !out_strides) { set_error("run_decode_fp4: NULL tensor"); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(q) || !aligned16(out) || (float_ws && !aligned16(float_ws))) { set_error("run_decode_fp4: tensors must be 16-byte aligned"); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i) {
    if (q_strides[i] % 8 || out_strides[i] % 8) {
      set_error("run_decode_fp4: q/out strides must be multiples of 8 elements");
      return BSKV_ERR_INVALID_ARG;
    }
  }
  const bool grid = meta_word(plan, H_GRID) > 0;  // some request has a token
  if (grid)
    if (bskv_status s = check_fp4_cache("run_decode_fp4", kv_codes, codes_strides, kv_scales, scales_strides)) return s;
  Fp4DecodeParams dp{};
  dp.meta = plan->meta_dev;
  dp.q = q; dp.q_s0 = q_strides[0]; dp.q_s1 = q_strides[1];
  if (grid) {
    dp.codes = static_cast<const uint8_t*>(kv_codes);
    dp.c_s0 = codes_strides[0]; dp.c_s1 = codes_strides[1]; dp.c_s2 = codes_strides[2]; dp.c_s3 = codes_strides[3];
    dp.scales = static_cast<const uint8_t*>(kv_scales);
    dp.s_s0 = scales_strides[0]; dp.s_s1 = scales_strides[1]; dp.s_s2 = scales_strides[2];
  }
  dp.out = out; dp.o_s0 = out_strides[0]; dp.o_s1 = out_strides[1];
  dp.lse = lse;
  dp.num_kv_heads = plan->num_kv_heads;
  dp.group = plan->num_qo_heads / plan->num_kv_heads;
  dp.page_size = plan->page_size;
  dp.num_qo_heads = plan->num_qo_heads;
  const int slots = meta_word(plan, H_SLOTS);
  dp.ws_o = static_cast<float*>(float_ws);
  dp.ws_lse = slots ? reinterpret_cast<float*>(static_cast<uint8_t*>(float_ws) +
                                               ((size_t(slots) * dp.group * plan->head_dim * 4 + 255) & ~size_t(255)))
                    : nullptr;
  dp.off_workers = meta_word(plan, H_OFF_WORKERS);
  dp.off_chunks = meta_word(plan, H_OFF_CHUNKS);
  dp.off_merges = meta_word(plan, H_OFF_MERGES);
  dp.off_aux0 = meta_word(plan, H_OFF_AUX0);
  dp.off_aux1 = meta_word(plan, H_OFF_AUX1);
  dp.num_merges = meta_word(plan, H_MERGES);
  dp.num_workers = meta_word(plan, H_WORKERS);
  dp.scale_log2 = sm_scale_log2(sm_scale, plan->head_dim);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fused = grid && dp.num_merges > 0 && plan->max_merge_count <= kFusedMergeMaxPieces;
  if (fused) dp.counters = plan->counters_dev;
  if (grid) {
    const bskv_status s = plan->dtype == BSKV_BF16 ? launch_t<__nv_bfloat16>(plan, dp, st)
                                                   : launch_t<__half>(plan, dp, st);
    if (s) return s;
  }
  if (dp.num_merges == 0 || fused) return BSKV_OK;
  return launch_state_merge(plan, plan->meta_dev, dp.ws_o, dp.ws_lse, out, out_strides, lse,
                            dp.num_kv_heads, dp.group, st);
}
