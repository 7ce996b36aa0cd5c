// Split-KV pieces of a paged decode: the order in which a worker walks its chunks, the merge
// item of a unit, and the log-sum-exp merge of the pieces' partial states.
#pragma once

#include <math.h>

#include "common.cuh"

namespace bskv {
namespace dev {

// Merge `count` partial states of output rows row0..row0+nrows-1 (of slots
// first..first+count-1, slot_rows rows per slot) into out0 + r * out_stride and lse0[r];
// count == 0 writes zeros and -inf. One warp; a lane covers 4 values of every (128 / D)-th
// row, NI rows (2 NI for D = 64) per pass. The slots are loaded B at a time (all in flight
// together) and combined one by one in slot order (the result depends on neither B nor NI):
//   m' = max(m, lse_c), s = exp(m - m'), w = exp(lse_c - m'),
//   l' = l s + w, acc' = acc s + w o_c;  out = acc / l, lse = m + log(l),
// the log-sum-exp merge of attention states. Partials written by other SMs in the same
// launch are read through L2 (ld.global.cg).
template <typename T, int D, int B = 4, int NI = 4>
__device__ __forceinline__ void merge_rows(int lane, const float* ws_o, const float* ws_lse,
                                           int first, int count, int slot_rows, int row0,
                                           int nrows, T* out0, int64_t out_stride, float* lse0) {
  constexpr int RS = 128 / D;  // rows covered by one pass of the warp
  const int dl = (lane * 4) % D, rl = (lane * 4) / D;
  for (int rb = 0; rb < nrows; rb += NI * RS) {
    float m[NI], tot[NI];
    float4 acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      m[i] = -INFINITY;
      tot[i] = 0.f;
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c0 = 0; c0 < count; c0 += B) {
      float bl[B][NI];
      float4 bx[B][NI];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int64_t base = int64_t(first + c0 + j) * slot_rows + row0 + rb + rl;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (c0 + j < count && rb + rl + RS * i < nrows) {
            bl[j][i] = __ldcg(ws_lse + base + RS * i);
            bx[j][i] = __ldcg(reinterpret_cast<const float4*>(ws_o + (base + RS * i) * D + dl));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (c0 + j >= count || rb + rl + RS * i >= nrows) continue;
          const float mn = fmaxf(m[i], bl[j][i]);
          const float sc = m[i] == -INFINITY ? 0.f : expf(m[i] - mn);
          const float w = expf(bl[j][i] - mn);
          tot[i] = tot[i] * sc + w;
          acc[i].x = acc[i].x * sc + w * bx[j][i].x;
          acc[i].y = acc[i].y * sc + w * bx[j][i].y;
          acc[i].z = acc[i].z * sc + w * bx[j][i].z;
          acc[i].w = acc[i].w * sc + w * bx[j][i].w;
          m[i] = mn;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = rb + rl + RS * i;
      if (r >= nrows) continue;
      const float inv = count > 0 ? 1.f / tot[i] : 0.f;
      // two 4-byte stores: output strides need only be multiples of 2 elements
      uint32_t* dst = reinterpret_cast<uint32_t*>(out0 + r * out_stride + dl);
      dst[0] = MmaOp<T>::pack(acc[i].x * inv, acc[i].y * inv);
      dst[1] = MmaOp<T>::pack(acc[i].z * inv, acc[i].w * inv);
      if (lse0 && dl == 0) lse0[r] = count > 0 ? m[i] + logf(tot[i]) : -INFINITY;
    }
  }
}

// The order in which a worker walks its chunks c0..c1-1: its last chunk first, then the
// others in order. A unit cut between workers w and w+1 is the last chunk of w and the
// first of w+1, so both pieces are computed early and its merge is off the kernel's tail.
__device__ __forceinline__ int chunk_at(int c0, int c1, int k) {
  return c1 - c0 >= 2 ? (k == 0 ? c1 - 1 : c0 + k - 1) : c0 + k;
}

// Merge item (unit, first_slot, count) of `unit`; items are sorted by unit.
__device__ __forceinline__ int find_merge_item(const int32_t* merges, int n, int unit) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (merges[3 * mid] < unit) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

}  // namespace dev
}  // namespace bskv
