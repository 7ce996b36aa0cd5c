// Eviction from a paged cache by accumulated attention weight: which tokens stay, and the
// compaction of their rows.
//
// Selection. Per (request, kv head): the first `sink` and the last `recent` tokens stay, and of
// the others the k of highest score (NaN above everything, -0 = +0, the lowest slot among equals).
// Scores become 32-bit keys of the same order; three histogram passes (11, 11 and 10 bits) find
// the k-th largest key T, and one pass in slot order keeps the keys above T and the first ones
// equal to it. Counts are integers, so the result does not depend on the order of the atomics.
//
// Compaction. Kept tokens move to the front in their order: row j comes from slot kept[j] >= j.
// Within one cache it is done in place: rows are taken in waves of ascending j, every read of a
// wave before its first write (one barrier), and a later wave only reads slots above every slot
// written so far. A wave's rows therefore never meet, so column slices of the rows (64 bytes of
// K or of V of a head), the scores and the 4-bit scales each go through their waves on their own
// CTA. Into other pages there is nothing to order and the rows are split over CTAs too.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

struct EvictParams {
  const int32_t* meta;
  float* scores;
  int64_t w_s0, w_s1;  // floats: page, kv head
  int32_t* kept;
  int64_t total;       // kept tokens over all requests
  int off_req, off_src, off_src_ptr, off_dst, page_size, num_kv_heads;
  int sink, recent, in_place;
};

// {tokens, kept tokens, first of them in `kept`, first destination page entry}
__device__ __forceinline__ int4 request_of(const EvictParams& p, int b) {
  return __ldg(reinterpret_cast<const int4*>(p.meta + p.off_req) + b);
}

// ---------------------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelectKeys = 49152;  // keys that shared memory holds; longer ranges are read again

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes +0
  if (x != x) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the CTA of one value per thread; total in *sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = lane < kSelectWarps ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
  *sum = __shfl_sync(0xffffffffu, s, 31);
  __syncthreads();  // warp_sums may be written again
  return before + x - v;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int warp_sums[kSelectWarps], warp_eq[kSelectWarps];
  __shared__ uint32_t found_digit;
  __shared__ int found_rest;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 rq = request_of(p, b);
  const int L = rq.x, K = rq.y;
  int32_t* kept = p.kept + h * p.total + rq.z;
  if (K == L) {
    for (int j = tid; j < K; j += kSelectThreads) kept[j] = j;
    return;
  }
  const int first = p.sink, N = L - p.sink - p.recent, k = K - p.sink - p.recent;
  for (int j = tid; j < p.sink; j += kSelectThreads) kept[j] = j;
  for (int j = tid; j < p.recent; j += kSelectThreads) kept[K - p.recent + j] = L - p.recent + j;
  if (k == 0) return;
  const int32_t* pages = p.meta + p.off_src + __ldg(p.meta + p.off_src_ptr + b);
  const float* scores = p.scores + h * p.w_s1;
  const bool held = N <= kSelectKeys;
  auto load = [&](int i) {
    const int t = first + i, n = t / p.page_size;
    return order_key(scores[__ldg(pages + n) * p.w_s0 + (t - n * p.page_size)]);
  };
  if (held) {
    for (int i = tid; i < N; i += kSelectThreads) keys[i] = load(i);
    __syncthreads();
  }
  auto key = [&](int i) { return held ? keys[i] : load(i); };

  // digits of T from the top; `rest` of the keys that share the digits so far are at or above T
  uint32_t T = 0;
  int rest = k;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < N; i += kSelectThreads) {
      const uint32_t x = key(i);
      if (pass == 0 || (x ^ T) >> (shift + bits) == 0)
        atomicAdd(&hist[(x >> shift) & ((1u << bits) - 1)], 1);
    }
    __syncthreads();
    // thread i has the bins 2047 - 2 i and 2046 - 2 i: prefix sums run from the largest keys
    const int hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
    int sum;
    const int before = block_scan(hi + lo, warp_sums, &sum);
    if (before < rest && rest <= before + hi + lo) {
      const bool upper = rest <= before + hi;
      found_digit = uint32_t(kBins - 1 - 2 * tid - (upper ? 0 : 1));
      found_rest = rest - before - (upper ? 0 : hi);
    }
    __syncthreads();
    T |= found_digit << shift;
    rest = found_rest;
    __syncthreads();
  }

  // each warp takes a contiguous part of the range: counts, then places
  const int part = ((N + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int i0 = min(N, warp * part), i1 = min(N, i0 + part);
  int above = 0, equal = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t x = i < i1 ? key(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < i1 && x > T));
    equal += __popc(__ballot_sync(0xffffffffu, i < i1 && x == T));
  }
  if (lane == 0) {
    warp_sums[warp] = above;
    warp_eq[warp] = equal;
  }
  __syncthreads();
  int at = 0, eq = 0;
  for (int w = 0; w < warp; ++w) {
    at += warp_sums[w];
    eq += warp_eq[w];
  }
  at += first + min(eq, rest);
  const uint32_t below = (1u << lane) - 1;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t x = i < i1 ? key(i) : 0u;
    const uint32_t em = __ballot_sync(0xffffffffu, i < i1 && x == T);
    const bool stay = i < i1 && (x > T || (x == T && eq + __popc(em & below) < rest));
    const uint32_t sm = __ballot_sync(0xffffffffu, stay);
    if (stay) kept[at + __popc(sm & below)] = first + i;
    at += __popc(sm);
    eq += __popc(em);
  }
}

// ---------------------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;  // rows a thread holds between a wave's reads and its writes

// One column slice of a paged tensor's rows: `lanes` units per row (16, 4 or 2 bytes each).
struct Plane {
  uint8_t* base;
  int64_t s0, s_head, s_slot;  // bytes
  int unit, lanes;
};
constexpr int kMaxPlanes = 10;
struct MoveParams {
  EvictParams e;
  Plane plane[kMaxPlanes];
};

template <typename U>
__device__ __forceinline__ void move_plane(const EvictParams& p, const Plane& pl, int b, int h,
                                           int part, int parts) {
  const int4 rq = request_of(p, b);
  const int32_t* kept = p.kept + h * p.total + rq.z;
  const int32_t* src_pages = p.meta + p.off_src + __ldg(p.meta + p.off_src_ptr + b);
  const int32_t* dst_pages = p.meta + p.off_dst + rq.w;
  uint8_t* base = pl.base + h * pl.s_head;
  const int lane = threadIdx.x % pl.lanes, per = kMoveThreads / pl.lanes;
  const int wave = per * kMoveRows, ps = p.page_size;
  const int K = rq.y;
  if (p.in_place && K == rq.x) return;
  U x[kMoveRows];
  uint8_t* to[kMoveRows];
  for (int w = part * wave; w < K; w += parts * wave) {
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const int j = w + i * per + threadIdx.x / pl.lanes;
      to[i] = nullptr;
      if (j >= K) continue;
      const int s = __ldcg(kept + j);
      if (p.in_place && s == j) continue;
      const int sn = s / ps, dn = j / ps;
      x[i] = *reinterpret_cast<const U*>(base + __ldg(src_pages + sn) * pl.s0 + (s - sn * ps) * pl.s_slot + lane * sizeof(U));
      to[i] = base + __ldg(dst_pages + dn) * pl.s0 + (j - dn * ps) * pl.s_slot + lane * sizeof(U);
    }
    if (p.in_place) __syncthreads();  // every read of the wave before its first write
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i)
      if (to[i]) *reinterpret_cast<U*>(to[i]) = x[i];
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ MoveParams p,
                                                                  int planes) {
  const int pl = blockIdx.x % planes, part = blockIdx.x / planes, parts = gridDim.x / planes;
  const int h = blockIdx.y, b = blockIdx.z;
  const Plane& plane = p.plane[pl];
  if (plane.unit == 16) move_plane<uint4>(p.e, plane, b, h, part, parts);
  else if (plane.unit == 4) move_plane<uint32_t>(p.e, plane, b, h, part, parts);
  else move_plane<uint16_t>(p.e, plane, b, h, part, parts);
}

bskv_status run(const char* who, const bskv_plan* plan, float* scores, const int64_t* scores_strides,
                int32_t* kept, bool compact_scores, MoveParams& mp, int planes, cudaStream_t st) {
  if (!scores || !scores_strides || !kept || !aligned16(scores)) { set_error("%s: scores must be a 16-byte aligned tensor, and kept given", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i) {
    if (scores_strides[i] <= 0 || scores_strides[i] % 4) {
      set_error("%s: scores stride %d (%lld) must be a positive multiple of 4 elements", who, i, (long long)scores_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  EvictParams& e = mp.e;
  e.meta = plan->meta_dev;
  e.scores = scores; e.w_s0 = scores_strides[0]; e.w_s1 = scores_strides[1];
  e.kept = kept; e.total = plan->kept_total;
  e.off_req = meta_word(plan, H_OFF_CHUNKS);
  e.off_src_ptr = meta_word(plan, H_OFF_AUX0);
  e.off_src = meta_word(plan, H_OFF_AUX1);
  e.off_dst = plan->in_place ? e.off_src : meta_word(plan, H_OFF_WORKERS);
  e.page_size = plan->page_size; e.num_kv_heads = plan->num_kv_heads;
  e.sink = plan->sink; e.recent = plan->recent; e.in_place = plan->in_place;
  if (compact_scores)
    mp.plane[planes++] = Plane{reinterpret_cast<uint8_t*>(scores), 4 * e.w_s0, 4 * e.w_s1, 4, 4, 1};
  const int smem = int(sizeof(uint32_t)) * std::min(kSelectKeys, plan->longest);
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), size_t(smem), allowed,
                                 "evict: cudaFuncSetAttribute"))
    return s;
  evict_select_kernel<<<dim3(unsigned(plan->num_kv_heads), unsigned(plan->batch)), kSelectThreads, smem, st>>>(e);
  if (bskv_status s = cuda_check(cudaGetLastError(), "evict select launch")) return s;
  const int parts = plan->in_place ? 1 : plan->parts;
  evict_move_kernel<<<dim3(unsigned(planes * parts), unsigned(plan->num_kv_heads), unsigned(plan->batch)),
                      kMoveThreads, 0, st>>>(mp, planes);
  return cuda_check(cudaGetLastError(), "evict move launch");
}

bskv_status check_plan(const char* who, const bskv_plan* plan) {
  if (!plan || plan->kind != KIND_EVICT) { set_error("%s: not an eviction plan", who); return BSKV_ERR_INVALID_ARG; }
  if (!plan->meta_dev) { set_error("%s: plan not uploaded (bskv_plan_upload)", who); return BSKV_ERR_INVALID_ARG; }
  return BSKV_OK;
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_run_evict(const bskv_plan* plan, float* scores,
                                      const int64_t* scores_strides, int32_t compact_scores,
                                      void* kv_cache, const int64_t* kv_strides, int32_t* kept,
                                      void* stream) {
  BSKV_NVTX_RANGE("bskv_run_evict");
  const char* who = "run_evict";
  if (bskv_status s = check_plan(who, plan)) return s;
  if (plan->kept_total == 0) return BSKV_OK;
  if (!kv_cache || !kv_strides || !aligned16(kv_cache)) { set_error("%s: kv_cache must be a 16-byte aligned tensor", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 4; ++i) {
    if (kv_strides[i] <= 0 || kv_strides[i] % 8) {
      set_error("%s: kv stride %d (%lld elements) must be positive and 16-byte aligned", who, i, (long long)kv_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  MoveParams mp{};
  int planes = 0;
  for (int which = 0; which < 2; ++which)
    for (int col = 0; col < 2 * plan->head_dim; col += 64)
      mp.plane[planes++] = Plane{static_cast<uint8_t*>(kv_cache) + 2 * which * kv_strides[1] + col,
                                 2 * kv_strides[0], 2 * kv_strides[2], 2 * kv_strides[3], 16, 4};
  return run(who, plan, scores, scores_strides, kept, compact_scores != 0, mp, planes,
             static_cast<cudaStream_t>(stream));
}

extern "C" bskv_status bskv_run_evict_fp4(const bskv_plan* plan, float* scores,
                                          const int64_t* scores_strides, int32_t compact_scores,
                                          void* kv_codes, const int64_t* codes_strides,
                                          void* kv_scales, const int64_t* scales_strides,
                                          int32_t* kept, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_evict_fp4");
  const char* who = "run_evict_fp4";
  if (bskv_status s = check_plan(who, plan)) return s;
  if (plan->kept_total == 0) return BSKV_OK;
  if (bskv_status s = check_fp4_cache(who, kv_codes, codes_strides, kv_scales, scales_strides)) return s;
  MoveParams mp{};
  int planes = 0;
  const int blocks = plan->head_dim / kFp4Block;
  for (int which = 0; which < 2; ++which) {
    mp.plane[planes++] = Plane{static_cast<uint8_t*>(kv_codes) + which * codes_strides[1], codes_strides[0],
                               codes_strides[2], codes_strides[3], 16, plan->head_dim / 32};
    mp.plane[planes++] = Plane{static_cast<uint8_t*>(kv_scales) + which * scales_strides[1],
                               scales_strides[0], scales_strides[2], blocks, blocks, 1};
  }
  return run(who, plan, scores, scores_strides, kept, compact_scores != 0, mp, planes,
             static_cast<cudaStream_t>(stream));
}
