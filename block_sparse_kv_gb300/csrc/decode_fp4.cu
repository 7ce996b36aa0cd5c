// Paged-KV batch decode over a microscaled 4-bit cache, with split-KV and the LSE merge.
//
// Mathematics. K[j, d] = e_K[j, d] X[j, d / 32] with E2M1 codes e and power-of-two scales X
// (and V alike), so
//   q.k_j  = sum_blocks X_K[j, b] (sum_{d in b} q_d e_K[j, d])
//   o_d    = sum_j (p_j X_V[j, d / 32]) e_V[j, d]
// The codes are exact in f16, so both inner sums are f16 tensor-core products of the codes
// themselves: a key's scale multiplies the fp32 partial sum of its block, a value's scale is
// folded into the softmax weight. Queries in bf16 are made f16 by an exact power of two per
// head. Weight times scale, p_j X_V[j, b], is rounded to f16. The reference that weights are
// taken relative to (any reference gives the same softmax) is therefore not the largest logit but
// 2^10 below the largest product so far of the head, up to a factor 2^5: products down to 2^-24 of
// it keep f16's 11 bits, smaller ones are off by at most 2^-35 of it. It changes on the first tile
// and rarely after, so a tile has no reduction over its tokens, only a vote: a product past 2^15
// moves it, and so do weights that sum to 2^97, which tokens whose values are zero reach without one.
// Value scales so large that the weights would leave fp32's range at its lower end are taken relative to
// a power of two of the (request, kv head).
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
// 512 in 16 bits, so instructions issued per byte are what to save: converting and pairing 4-bit
// values keeps the ALU pipe busy for half to two thirds of the time. 64 requests of 512 to 4096
// tokens with 4 query heads per kv head take 40.6 us (4.0 TB/s), 8 of 131072 with 8 heads 238 us (4.8
// TB/s; with 16 heads 78 and 330 us). Blocks of zeros and the unit in the way of setting a reference cost
// 1.2 and 5 us of these. Without them 39.4 and 233 us were measured for what the loop is made of: a warp
// works on 32 tokens at a time, the second 16's products fill the first's waits (41.2 and 239 us with
// 16), and two stages are enough of a ring (three: 41.9 and 243 us).
// Each warp is a worker of its own over a range of one or more (request, kv
// head) units, with a private ring of 32-token tiles filled by 16-byte asynchronous copies
// (any page size and stride, no swizzle constraint on the page layout). A unit cut between
// workers is merged in the same launch as in the 16-bit decode, by the same code.
#include <math.h>

#include "cache_common.cuh"
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
constexpr int kStages = 2;

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
  int num_kv_heads, group, num_qo_heads;
  FastDiv heads, page_size;
  int off_workers, off_records, off_merges, off_aux1, num_merges, num_workers;
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
  float o[NT][Shape<D>::kBlocks][2][4];     // O^T accumulators
  float ref[2 * NT], l[2 * NT], c[2 * NT];  // exponent reference, sum, logit scale (base 2, > 0)
  int unit;                                 // value scales count relative to 2^unit >= 1; -1: no tokens yet
};

// Up to 4 query heads per kv head (NT = 0): column n of the products is head n / 2, so that a lane
// has one head, t. In O^T = V^T P^T the two columns of a head take the even and the odd values: the
// k-pair of the A operand is (value 2i, value 2i + 1) of one token, as the codes lie in a byte, and
// the B operand holds the weight in the half of its column's parity and zero in the other. That
// needs no pairing of two tokens' nibbles and wastes no column.
template <int D>
struct State<D, 0> {
  uint32_t q[Shape<D>::kBlocks][4];
  float o[Shape<D>::kBlocks][4];  // values 32 b + 4 g .. + 3 of head t
  float ref, l, c;
  int unit;
};

// Scale (base 2, > 0) of a head's logits; `back` is the power of two its query was divided by. Above 0
// even where the product is not: a masked token's -inf times 0 would be NaN.
__device__ __forceinline__ float logit_scale(float scale_log2, float back) {
  return fmaxf(fabsf(scale_log2) * back, 0x1p-149f);
}

template <typename T, int D, int NT>
__device__ __forceinline__ void load_q(const Fp4DecodeParams& p, int b, int kvh, int lane,
                                       State<D, NT>& s) {
  constexpr int NB = Shape<D>::kBlocks;
  const int g = lane >> 2, t = lane & 3;
  s.unit = -1;
  // a column without a head keeps the reference +inf: its weights are 0 and it asks for nothing
  if constexpr (NT == 0) {
    const float back = load_q_f16<T, NB>(
        static_cast<const T*>(p.q) + b * p.q_s0 + (int64_t(kvh) * p.group + (g >> 1)) * p.q_s1,
        (g >> 1) < p.group, p.scale_log2 < 0.f, lane, s.q);
    s.c = logit_scale(p.scale_log2, __shfl_sync(0xffffffffu, back, 8 * t));
    s.ref = t < p.group ? -INFINITY : INFINITY;
    s.l = 0.f;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) s.o[blk][0] = s.o[blk][1] = s.o[blk][2] = s.o[blk][3] = 0.f;
    return;
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + g;
      const float back = load_q_f16<T, NB>(
          static_cast<const T*>(p.q) + b * p.q_s0 + (int64_t(kvh) * p.group + h) * p.q_s1,
          h < p.group, p.scale_log2 < 0.f, lane, s.q[nt]);
      // columns 2t and 2t + 1 belong to the heads of lanes 8t and 8t + 4
      s.c[2 * nt] = logit_scale(p.scale_log2, __shfl_sync(0xffffffffu, back, 8 * t));
      s.c[2 * nt + 1] = logit_scale(p.scale_log2, __shfl_sync(0xffffffffu, back, 8 * t + 4));
    }
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      s.ref[j] = 8 * (j >> 1) + 2 * t + (j & 1) < p.group ? -INFINITY : INFINITY;
      s.l[j] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 8; ++i) s.o[nt][blk][i >> 2][i & 3] = 0.f;
  }
}

// A lane's sum of weights of one step (at most 4 tokens) past this calls for a new reference. A request
// has at most 2^30 tokens, 16 or more of them a step, so the sum over the steps and the 8 lanes of a
// head stays below 2^127.
constexpr float kMaxAdd = 0x1p97f;

// What 16 H tokens ask of a head's reference, a lane giving 2 H logits (base 2) and the exponents f of
// the tokens' largest scales (-inf without one): the largest logit, and of weight times scale.
struct Need {
  float top, product;
};
template <int N>
__device__ __forceinline__ Need need_of(const float (&v)[N], const float (&f)[N]) {
  Need n{v[0], v[0] + f[0]};
#pragma unroll
  for (int i = 1; i < N; ++i) {
    n.top = fmaxf(n.top, v[i]);
    n.product = fmaxf(n.product, v[i] + f[i]);
  }
  return Need{max_over_rows(n.top), max_over_rows(n.product)};
}
// By how many powers of two the unit has to grow so that a reference 2^10 below the head's largest
// product stands at most 2^40 above its largest weight so far, which is 2^-40 of the old reference or
// more.
__device__ __forceinline__ float unit_growth(float ref, const Need& n, int unit) {
  const float x = n.product - 10.f - max(unit, 0) - fmaxf(n.top, ref - 40.f);
  return x > 40.f ? ceilf(x) : 0.f;
}
// The reference 2^10 below the largest product, relative to the unit, and at most 2^94 below the largest
// weight. It falls only with the unit, by which all heads' products have become smaller, and no further
// than leaves the weights so far, whose sum in the lane is l, below 2^94. Returns the square root of what
// that sum shrinks by, or grows: a factor of up to 2^-134 matters, to weights of 2^94.
__device__ __forceinline__ float move_ref(float& ref, const Need& n, int unit, int grown, float l) {
  float least = ref;
  if (grown > 0) least = fminf(ref, fmaxf(ref - grown, ref + float(exponent_of(max_over_rows(l)) + 1 - 94)));
  const float to = fmaxf(least, fmaxf(n.product - 10.f - unit, n.top - 94.f));
  const float root = fast_exp2(0.5f * (ref - to));
  ref = to;
  return root;
}
// The warp's unit grows by the most that a lane asks for; returns by how much.
__device__ __forceinline__ int grow_unit(int& unit, float growth) {
  const int by = __reduce_max_sync(0xffffffffu, int(growth));
  unit = max(unit, 0) + by;
  return by;
}

template <int D, int NT, int N>
__device__ __forceinline__ void move_refs(State<D, NT>& s, const float (&x)[NT][2][N], const float (&f)[N]) {
  Need need[2 * NT];
  float growth = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[j >> 1][j & 1][i] * s.c[j];
    need[j] = need_of(v, f);
    growth = fmaxf(growth, unit_growth(s.ref[j], need[j], s.unit));
  }
  const int grown = grow_unit(s.unit, growth);
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const float root = move_ref(s.ref[j], need[j], s.unit, grown, s.l[j]), root_o = root * pow2(-grown);
    s.l[j] = s.l[j] * root * root;
#pragma unroll
    for (int blk = 0; blk < Shape<D>::kBlocks; ++blk)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float& a = s.o[j >> 1][blk][i][j & 1];
        float& b = s.o[j >> 1][blk][i][(j & 1) + 2];
        a = a * root * root_o;
        b = b * root * root_o;
      }
  }
}

// The lane's value scales relative to the unit.
template <int NB, int N>
__device__ __forceinline__ void to_unit(int unit, float (&sv)[N][NB]) {
  const float u = pow2(-unit);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) sv[i][blk] *= u;
}

// Largest exponent of the scales of each token's value blocks, -inf where all values are zero or NaN. A
// block of zeros gives nothing whatever its scale, which may stand far above the others': it becomes 0.
// Row i of the lane is r0 + 8 i, its block blk at part blk ^ kx; the four lanes of a row look at a block
// each.
template <int D, int N>
__device__ __forceinline__ void scale_exponents(const uint8_t* st, int r0, int kx, float (&sv)[N][Shape<D>::kBlocks],
                                                float (&f)[N]) {
  using Sh = Shape<D>;
  const int quad = threadIdx.x & 28, mine = threadIdx.x & (Sh::kBlocks - 1);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint4 c = *reinterpret_cast<const uint4*>(st + Sh::kV + (r0 + 8 * i) * Sh::kRow + ((mine ^ kx) << 4));
    const uint32_t zeros = __ballot_sync(0xffffffffu, ((c.x | c.y | c.z | c.w) & 0x77777777u) == 0) >> quad;
    float big = 0.f;
#pragma unroll
    for (int blk = 0; blk < Sh::kBlocks; ++blk) {
      if ((zeros >> blk & 1u) && sv[i][blk] == sv[i][blk]) sv[i][blk] = 0.f;
      big = fmaxf(big, sv[i][blk]);
    }
    f[i] = big > 0.f ? float(exponent_of(big)) : -INFINITY;
  }
}

// 16 H tokens from row `first` of a tile in shared memory on; with WHOLE false, rows >= valid lie
// past the chunk (valid > first). Row i of a lane is first + g + 8 i.
template <int D, int NT, bool WHOLE, int H>
__device__ __forceinline__ void some_tokens(const uint8_t* st, int first, int valid, int lane, State<D, NT>& s) {
  using Sh = Shape<D>;
  using Mma = MmaOp<__half>;
  constexpr int NB = Sh::kBlocks, N = 2 * H;
  const int g = lane >> 2, t = lane & 3, r0 = first + g;
  const int kx = (g >> Sh::kSwzShift) & (Sh::kParts - 1);
  const int vx = ((2 * t) >> Sh::kSwzShift) & (Sh::kParts - 1);
  float x[NT][2][N];  // q.k of columns 2t and 2t + 1
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float s0[NB], s1[NB];
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r0 + 8 * i), s0);
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r0 + 8 * i + 8), s1);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint8_t* at = st + ((blk ^ kx) << 4) + 4 * t + (r0 + 8 * i) * Sh::kRow;
      uint32_t a0[4], a1[4];
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at), a0);
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at + 8 * Sh::kRow), a1);
      const uint32_t f0[4] = {a0[0], a1[0], a0[1], a1[1]}, f1[4] = {a0[2], a1[2], a0[3], a1[3]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        Mma::run(acc, f0, s.q[nt][blk][0], s.q[nt][blk][1]);
        Mma::run(acc, f1, s.q[nt][blk][2], s.q[nt][blk][3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[nt][e][i] = blk ? fmaf(acc[e], s0[blk], x[nt][e][i]) : acc[e] * s0[blk];
          x[nt][e][i + 1] = blk ? fmaf(acc[e + 2], s1[blk], x[nt][e][i + 1]) : acc[e + 2] * s1[blk];
        }
      }
    }
    if constexpr (!WHOLE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (r0 + 8 * i >= valid) x[nt][e][i] = -INFINITY;
          if (r0 + 8 * i + 8 >= valid) x[nt][e][i + 1] = -INFINITY;
        }
    }
  }
  // Weights relative to the reference, times the value scales, as f16 pairs of two heads. Products
  // up to 2^15 are safe in f16; the first tokens, and later ones with a larger product, set it. Where the
  // unit is above 1 all tokens take the second way: a branch around the factor in the first costs ordinary
  // caches 5 to 7 % (64 requests of 512 to 4096 tokens 41.7 us, 8 of 131072 with 8 heads 249).
  float sv[N][NB];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t w = scale_word<D>(st + Sh::kVs, r0 + 8 * i);
    if constexpr (!WHOLE) w = r0 + 8 * i < valid ? w : 0u;
    scales_of<NB>(w, sv[i]);
  }
  uint32_t pp[NT][NB][N];
  float add[2 * NT];
  auto weigh = [&]() {
    __half2 top = __float2half2_rn(0.f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      add[2 * nt] = add[2 * nt + 1] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float e[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          e[k] = fast_exp2(fmaf(x[nt][k][i], s.c[2 * nt + k], -s.ref[2 * nt + k]));
          add[2 * nt + k] += e[k];
        }
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          const uint32_t w = pack_half2(e[0] * sv[i][blk], e[1] * sv[i][blk]);
          pp[nt][blk][i] = w;
          top = __hmax2(top, *reinterpret_cast<const __half2*>(&w));
        }
      }
    }
    float most = add[0];
#pragma unroll
    for (int j = 1; j < 2 * NT; ++j) most = fmaxf(most, add[j]);
    return most > kMaxAdd || __hgt(__hmax(__low2half(top), __high2half(top)), __float2half(32768.f));
  };
  const bool over = weigh();
  if (__any_sync(0xffffffffu, over || s.unit != 0)) {
    float f[N];
    scale_exponents<D>(st, r0, kx, sv, f);
    move_refs<D, NT>(s, x, f);
    to_unit(s.unit, sv);
    weigh();
  }
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) s.l[j] += add[j];
  // O^T += V^T P^T, 16 tokens a product
  const uint8_t* row = st + Sh::kV + (first + 2 * t) * Sh::kRow + 2 * g;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint8_t* at = row + ((blk ^ vx) << 4) + 16 * h * Sh::kRow;
      const uint32_t h0 = *reinterpret_cast<const uint16_t*>(at);
      const uint32_t h1 = *reinterpret_cast<const uint16_t*>(at + Sh::kRow);
      const uint32_t h2 = *reinterpret_cast<const uint16_t*>(at + 8 * Sh::kRow);
      const uint32_t h3 = *reinterpret_cast<const uint16_t*>(at + 9 * Sh::kRow);
      const uint32_t even = __byte_perm(h0, h2, 0x5410), odd = __byte_perm(h1, h3, 0x5410);
      uint32_t lo[4], hi[4];  // rows g / g + 8 of the two products: values 4g + {0, 1} and {2, 3}
      cvt_e2m1x8(nibbles(even, odd << 4), lo);
      cvt_e2m1x8(nibbles(even >> 4, odd), hi);
      const uint32_t a[2][4] = {{lo[0], hi[0], lo[2], hi[2]}, {lo[1], hi[1], lo[3], hi[3]}};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t b0 = movmatrix(pp[nt][blk][2 * h]), b1 = movmatrix(pp[nt][blk][2 * h + 1]);
        Mma::run(s.o[nt][blk][0], a[0], b0, b1);
        Mma::run(s.o[nt][blk][1], a[1], b0, b1);
      }
    }
}

// A pair of weights' halves into the half of the lane's column parity, zero elsewhere: byte
// selectors for the low (e = 0) and the high weight.
__device__ __forceinline__ uint32_t half_select(int e, int parity) {
  return parity ? (e ? 0x3244u : 0x1044u) : (e ? 0x4432u : 0x4410u);
}

// some_tokens for up to 4 query heads per kv head.
template <int D, bool WHOLE, int H>
__device__ __forceinline__ void some_tokens4(const uint8_t* st, int first, int valid, int lane, State<D, 0>& s) {
  using Sh = Shape<D>;
  using Mma = MmaOp<__half>;
  constexpr int NB = Sh::kBlocks, N = 2 * H;
  const int g = lane >> 2, t = lane & 3, r0 = first + g;
  const int kx = (g >> Sh::kSwzShift) & (Sh::kParts - 1);
  float x[N];  // q.k of the lane's tokens with head t
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float s0[NB], s1[NB];
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r0 + 8 * i), s0);
    scales_of<NB>(scale_word<D>(st + Sh::kKs, r0 + 8 * i + 8), s1);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint8_t* at = st + ((blk ^ kx) << 4) + 4 * t + (r0 + 8 * i) * Sh::kRow;
      uint32_t a0[4], a1[4];
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at), a0);
      cvt_e2m1x8(*reinterpret_cast<const uint32_t*>(at + 8 * Sh::kRow), a1);
      const uint32_t f0[4] = {a0[0], a1[0], a0[1], a1[1]}, f1[4] = {a0[2], a1[2], a0[3], a1[3]};
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      Mma::run(acc, f0, s.q[blk][0], s.q[blk][1]);
      Mma::run(acc, f1, s.q[blk][2], s.q[blk][3]);
      x[i] = blk ? fmaf(acc[0], s0[blk], x[i]) : acc[0] * s0[blk];
      x[i + 1] = blk ? fmaf(acc[2], s1[blk], x[i + 1]) : acc[2] * s1[blk];
    }
    if constexpr (!WHOLE) {
      if (r0 + 8 * i >= valid) x[i] = -INFINITY;
      if (r0 + 8 * i + 8 >= valid) x[i + 1] = -INFINITY;
    }
  }
  float sv[N][NB];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t w = scale_word<D>(st + Sh::kVs, r0 + 8 * i);
    if constexpr (!WHOLE) w = r0 + 8 * i < valid ? w : 0u;
    scales_of<NB>(w, sv[i]);
  }
  uint32_t pw[N][NB / 2];  // weight times scale of blocks 2 n and 2 n + 1
  float add;
  auto weigh = [&]() {
    __half2 top = __float2half2_rn(0.f);
    add = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = fast_exp2(fmaf(x[i], s.c, -s.ref));
      add += e;
#pragma unroll
      for (int n = 0; n < NB / 2; ++n) {
        pw[i][n] = pack_half2(e * sv[i][2 * n], e * sv[i][2 * n + 1]);
        top = __hmax2(top, *reinterpret_cast<const __half2*>(&pw[i][n]));
      }
    }
    return add > kMaxAdd || __hgt(__hmax(__low2half(top), __high2half(top)), __float2half(32768.f));
  };
  const bool over = weigh();
  if (__any_sync(0xffffffffu, over || s.unit != 0)) {
    float f[N], v[N];
    scale_exponents<D>(st, r0, kx, sv, f);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i] * s.c;
    const Need need = need_of(v, f);
    const int grown = grow_unit(s.unit, unit_growth(s.ref, need, s.unit));
    const float root = move_ref(s.ref, need, s.unit, grown, s.l), root_o = root * pow2(-grown);
    s.l = s.l * root * root;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 4; ++i) s.o[blk][i] = s.o[blk][i] * root * root_o;
    to_unit(s.unit, sv);
    weigh();
  }
  s.l += add;
  // O^T += V^T P^T, 8 tokens a product: lane (g, t) gives tokens t and t + 4 of head g / 2
  const uint32_t sel0 = half_select(0, g & 1), sel1 = half_select(1, g & 1);
  const int vx = (t >> Sh::kSwzShift) & (Sh::kParts - 1), vx4 = ((t + 4) >> Sh::kSwzShift) & (Sh::kParts - 1);
  const uint8_t* row = st + Sh::kV + (first + t) * Sh::kRow + 2 * g;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int n = 0; n < NB / 2; ++n) {
      const uint32_t p0 = __shfl_sync(0xffffffffu, pw[i][n], 4 * t + (g >> 1));
      const uint32_t p4 = __shfl_sync(0xffffffffu, pw[i][n], 4 * (t + 4) + (g >> 1));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int blk = 2 * n + e;
        const uint8_t* at = row + 8 * i * Sh::kRow;
        uint32_t a[4];
        cvt_e2m1x4(*reinterpret_cast<const uint16_t*>(at + ((blk ^ vx) << 4)), a[0], a[1]);
        cvt_e2m1x4(*reinterpret_cast<const uint16_t*>(at + 4 * Sh::kRow + ((blk ^ vx4) << 4)), a[2], a[3]);
        Mma::run(s.o[blk], a, __byte_perm(p0, 0u, e ? sel1 : sel0), __byte_perm(p4, 0u, e ? sel1 : sel0));
      }
    }
}

// Normalise a finished chunk and write it to out / lse (slot < 0) or as a partial state.
template <typename T, int D>
__device__ __forceinline__ void put_head(const Fp4DecodeParams& p, int b, int kvh, int slot, int h, int d, float4 v) {
  using Mma = MmaOp<T>;
  if (slot >= 0) {
    *reinterpret_cast<float4*>(p.ws_o + (int64_t(slot) * p.group + h) * D + d) = v;
  } else {
    T* dst = static_cast<T*>(p.out) + b * p.o_s0 + (int64_t(kvh) * p.group + h) * p.o_s1 + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(Mma::pack(v.x, v.y), Mma::pack(v.z, v.w));
  }
}
__device__ __forceinline__ void put_lse(const Fp4DecodeParams& p, int b, int kvh, int slot, int h, float lse) {
  if (slot >= 0) p.ws_lse[int64_t(slot) * p.group + h] = lse;
  else if (p.lse) p.lse[int64_t(b) * p.num_qo_heads + kvh * p.group + h] = lse;
}

template <typename T, int D, int NT>
__device__ __forceinline__ void finish(const Fp4DecodeParams& p, int b, int kvh, int slot, int lane,
                                       State<D, NT>& s) {
  constexpr int NB = Shape<D>::kBlocks;
  const int g = lane >> 2, t = lane & 3;
  const float u = pow2(s.unit);
  if constexpr (NT == 0) {
    const float l = sum_over_rows(s.l), inv = 1.f / l;
    if (t >= p.group) return;
    if (g == 0) put_lse(p, b, kvh, slot, t, (s.ref + __log2f(l)) * kLn2);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
      put_head<T, D>(p, b, kvh, slot, t, 32 * blk + 4 * g,
                     make_float4(s.o[blk][0] * inv * u, s.o[blk][1] * inv * u, s.o[blk][2] * inv * u, s.o[blk][3] * inv * u));
  } else {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int h = 8 * (j >> 1) + 2 * t + (j & 1), e = j & 1;
      const float l = sum_over_rows(s.l[j]), inv = 1.f / l;
      if (h >= p.group) continue;
      if (g == 0) put_lse(p, b, kvh, slot, h, (s.ref[j] + __log2f(l)) * kLn2);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        const auto& o = s.o[j >> 1][blk];
        put_head<T, D>(p, b, kvh, slot, h, 32 * blk + 4 * g,
                       make_float4(o[0][e] * inv * u, o[0][e + 2] * inv * u, o[1][e] * inv * u, o[1][e + 2] * inv * u));
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
  const int c0 = __ldg(p.meta + p.off_workers + w), nck = __ldg(p.meta + p.off_workers + w + 1) - c0;
  const int32_t* records = p.meta + p.off_records + c0 * kWalkWords;
  PageWalk walk(records, nck, p.meta + p.off_aux1, p.heads, p.page_size, lane);

  // Eight lanes copy a group of 8 tokens: row `sub / kParts` and every kRows-th after it, part
  // `sub % kParts` of each (XORed as swizzled), and the first of them its 16-byte pieces of scales.
  // What the addresses add to the group's own offset, kept by lane (tok - win) / 8 + j, is fixed.
  constexpr int kRows = 8 / Sh::kParts;
  constexpr int kPieces = 8 * Sh::kBlocks / 16;  // of a group's K scales
  const int j = lane >> 3, sub = lane & 7, which = (sub / kPieces) & 1, chunk = sub % kPieces;
  const uint8_t* k_lane = p.codes + sub / Sh::kParts * p.c_s3 + sub % Sh::kParts * 16;
  const uint8_t* s_lane = p.scales + which * p.s_s1 + chunk * 16;
  const int64_t step = kRows * p.c_s3;
  const uint32_t to_lane = smem_u32(ring + (8 * j + sub / Sh::kParts) * Sh::kRow + sub % Sh::kParts * 16);
  const uint32_t s_to_lane =
      smem_u32(ring + Sh::kKs + which * kTile * Sh::kBlocks + 8 * j * Sh::kBlocks + chunk * 16);
  int64_t c_off = 0, s_off = 0;
  auto issue = [&](int stage) {
    if (walk.live()) {
      if (walk.enter()) {
        c_off = walk.page * p.c_s0 + walk.kvh * p.c_s2 + walk.slot * p.c_s3;
        s_off = walk.page * p.s_s0 + walk.kvh * p.s_s2 + walk.slot * Sh::kBlocks;
      }
      const uint8_t* from = k_lane + walk.of_group(c_off, 8 * j);
      const uint8_t* s_from = s_lane + walk.of_group(s_off, 8 * j);
      if (walk.has(8 * j)) {
        const uint32_t to = to_lane + stage * Sh::kStage;
#pragma unroll
        for (int i = 0; i < Sh::kParts; ++i) {
          cp_async_16_at((to ^ (i << 4)) + i * kRows * Sh::kRow, from);
          cp_async_16_at((to ^ (i << 4)) + i * kRows * Sh::kRow + Sh::kV, from + p.c_s1);
          from += step;
        }
        if (sub < 2 * kPieces) cp_async_16_at(s_to_lane + stage * Sh::kStage, s_from);
      }
      walk.advance();
    }
    cp_async_commit();
  };

  for (int i = 0; i < kStages - 1; ++i) issue(i);

  State<D, NT> s;
  int done = 0, first_merge = -1, last_merge = -1;  // chunks whose units this worker merges
  for (int k = 0; k < nck; ++k) {
    const WalkChunk ch = walk_chunk(records, k);
    int kvh;
    const int b = p.heads.divmod(ch.unit, kvh);
    load_q<T, D, NT>(p, b, kvh, lane, s);
    for (int at = ch.begin; at < ch.end; at += kTile, ++done) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // the tile is there for every lane, and the stage refilled next is free
      issue((done + kStages - 1) % kStages);
      const uint8_t* st = ring + (done % kStages) * Sh::kStage;
      constexpr int H = NT == 2 ? 1 : 2;
      const int valid = ch.end - at;
      if (valid >= kTile) {
#pragma unroll 1
        for (int r = 0; r < kTile; r += 16 * H) {
          if constexpr (NT == 0) some_tokens4<D, true, H>(st, r, kTile, lane, s);
          else some_tokens<D, NT, true, H>(st, r, kTile, lane, s);
        }
      } else {
#pragma unroll 1
        for (int r = 0; r < valid; r += 16) {
          if constexpr (NT == 0) some_tokens4<D, false, 1>(st, r, valid, lane, s);
          else some_tokens<D, NT, false, 1>(st, r, valid, lane, s);
        }
      }
    }
    finish<T, D, NT>(p, b, kvh, ch.slot, lane, s);
    if (ch.slot >= 0 && p.counters) {
      // The last of the unit's chunks to finish merges all of them (release / acquire through
      // lane 0's atomic, the other lanes' writes ordered before it by the __syncwarp). Only the
      // first and the last chunk of a worker are pieces of a unit. The merges come after the loop:
      // a call inside it costs the loop its registers.
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomic_add_acq_rel(p.counters + ch.item, 1) == ch.pieces - 1;
      if (__shfl_sync(0xffffffffu, last, 0)) (k == 0 ? first_merge : last_merge) = k;
    }
  }
  cp_async_wait<0>();
  if (p.counters) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int k = i ? last_merge : first_merge;
      if (k < 0) continue;
      const WalkChunk ch = walk_chunk(records, k);
      merge_unit<T, D>(p, lane, ch.unit, ch.first_slot, ch.pieces);
      if (lane == 0) p.counters[ch.item] = 0;  // ready for the next run
    }
    // Units without tokens are zero-filled by the workers in turn.
#pragma unroll 1
    for (int i = w; i < p.num_merges; i += P)
      if (merges[3 * i + 2] == 0) merge_unit<T, D>(p, lane, merges[3 * i], 0, 0);
  }
}

template <typename T, int D, int NT>
bskv_status launch(const bskv_plan* plan, const Fp4DecodeParams& dp, cudaStream_t st) {
  const size_t smem = size_t(kWarps) * kStages * Shape<D>::kStage;
  auto kern = decode_fp4_kernel<T, D, NT>;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "decode_fp4: cudaFuncSetAttribute")) return s;
  kern<<<meta_word(plan, H_GRID), kWarps * 32, smem, st>>>(dp);
  return cuda_check(cudaGetLastError(), "decode_fp4 kernel launch");
}

template <typename T>
bskv_status launch_t(const bskv_plan* plan, const Fp4DecodeParams& dp, cudaStream_t st) {
  const int tiles = fp4_column_tiles(dp.group);
  if (plan->head_dim == 128)
    return tiles == 0 ? launch<T, 128, 0>(plan, dp, st) : tiles == 1 ? launch<T, 128, 1>(plan, dp, st) : launch<T, 128, 2>(plan, dp, st);
  return tiles == 0 ? launch<T, 64, 0>(plan, dp, st) : tiles == 1 ? launch<T, 64, 1>(plan, dp, st) : launch<T, 64, 2>(plan, dp, st);
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
  dp.heads = FastDiv(plan->num_kv_heads);
  dp.page_size = FastDiv(plan->page_size);
  dp.num_qo_heads = plan->num_qo_heads;
  const int slots = meta_word(plan, H_SLOTS);
  dp.ws_o = static_cast<float*>(float_ws);
  dp.ws_lse = slots ? reinterpret_cast<float*>(static_cast<uint8_t*>(float_ws) +
                                               ((size_t(slots) * dp.group * plan->head_dim * 4 + 255) & ~size_t(255)))
                    : nullptr;
  dp.off_workers = meta_word(plan, H_OFF_WORKERS);
  dp.off_records = plan->walk_records;
  dp.off_merges = meta_word(plan, H_OFF_MERGES);
  dp.off_aux1 = meta_word(plan, H_OFF_AUX1);
  dp.num_merges = meta_word(plan, H_MERGES);
  dp.num_workers = meta_word(plan, H_WORKERS);
  dp.scale_log2 = sm_scale_log2(sm_scale, plan->head_dim);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fused = grid && dp.num_merges > 0 && plan->max_merge_count <= kFp4FusedPieces;
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
