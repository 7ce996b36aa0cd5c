// Decode over chosen blocks of a paged cache: each (query, kv head) row attends to its own list.
//
// Mathematics. For query t, kv head h and the group's query heads, over the tokens j <= position of t that
// lie in a listed block (a page): out = sum_j softmax_j(scale q.k_j) v_j, lse = log sum_j exp(scale q.k_j),
// in one pass with a running maximum and sum.
//
// Bound by reading K and V of the listed blocks: a block of one head is a piece of page_size * D 16-bit
// values, wherever its page lies. One CTA per SM, eight warps with a ring of copies each, up to 192 KB in flight.
// The up to 16 query heads of a group are the M = 16 rows of mma.sync m16n8k16 against 16 tokens at a time. The
// weights go into the product with V as sums of two 16-bit values: of up to eight heads both parts are rows of one
// product, more heads take two.
//
// Split. The lists' lengths are known on the GPU only, so the cut is made in places: the rows' lists of top_k blocks
// follow one another in steps of 16 tokens (or pages of 8), and each team of 1, 2, 4 or 8 warps takes an equal run of
// them; a run covers the same fraction of a row's actual list (place f stands for step f n / top_k of a list of
// n blocks), so that short lists are cut as evenly as full ones. The warps of a team share each row of its run
// in equal parts and join their states in shared memory; a row that lies in several runs leaves their states in the
// float workspace, and the team that finishes its last piece joins them in the same launch, in piece order.
// A piece costs a warp about 4 us beside its tiles, which is why the team's size matters (1, 2, 4, 8 warps; us): 64
// requests, 8 kv heads, 64 blocks of 16 tokens 56.3, 50.3, 47.9, 47.7 (floor 40.2); 300 with 8 blocks 29.2, 31.0, 36.9,
// 56.8 (23.5); 32 with 32 blocks of 64 and 8 query heads per kv head 65.3, 55.0, 50.4, 48.3 (40.2); one with 128
// blocks 51.3, 18.1, 9.8, 9.1. The plan's rule is at blocks_team().
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "cache_common.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kTile = 16;  // tokens per stage
constexpr int kWarps = kBlocksWarps;
constexpr int kPanel = kTile * 128;  // 16 rows of 64 16-bit values, swizzled

struct BlocksParams {
  const void* q;
  int64_t q_s0, q_s1;
  void* out;
  int64_t o_s0, o_s1;
  float* lse;
  const int32_t *blocks, *batch_indices, *positions, *kv_indptr, *kv_indices;
  float *ws_o, *ws_lse;
  int* counters;   // per row: finished pieces
  int num_rows, top_k, team, workers, per_worker;
  int steps, row_places, places;  // steps of a block; places of a row: its steps and what a piece costs; of all rows
  int group, num_qo_heads, batch, num_pages;
  FastDiv heads, page_size, by_row, by_worker, by_steps;
  float scale_log2;
  StatusArgs st;
};

template <int D, int STAGES>
struct Ring {
  static constexpr int kTileBytes = (D / 64) * kPanel;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBytes = STAGES * kStageBytes;
};

// What the copying side tells the computing side about a stage.
struct StageInfo {
  int row;      // (query, kv head)
  int valid;    // tokens of its two groups of eight that are attended to: low and high half word
  int flags;    // 1: first tile of a piece, 2: last
};
constexpr int kFirst = 1, kLast = 2;

// Pieces of a row: those of the teams from `first` to `last`.
struct Pieces {
  int first, last;
};
__device__ __forceinline__ Pieces pieces_of(const BlocksParams& p, int row) {
  return Pieces{p.by_worker.div(row * p.row_places), p.by_worker.div(row * p.row_places + p.top_k * p.steps - 1)};
}

// A warp's way through its share of its team's run: row by row, 32 list entries at a time, one lane each.
struct Walk {
  const BlocksParams& p;
  int place, end;       // the team's places that are to come
  int member, lane;
  // the piece: this warp's steps [from, to) of the row's list, entries from `at` on are to come
  int row, from, to, at;
  int start, pos;       // of the row's request
  bool fresh;           // no tile of the piece has been given out
  // the window of up to 32 entries: lane i holds entry i's page and its attended slots [begin, end_slot)
  int page, begin, end_slot;
  uint32_t todo;        // entries that are not given out yet
  int entry, slot;      // the one being given out, and its next slot

  __device__ __forceinline__ Walk(const BlocksParams& p_, int worker, int member_, int lane_)
      : p(p_), place(worker * p_.per_worker), end(min(p_.places, place + p_.per_worker)), member(member_), lane(lane_), todo(0), entry(-1) {
    open();
  }
  __device__ __forceinline__ bool live() const { return row >= 0; }
  // The next piece, if there is one.
  __device__ __forceinline__ void open() {
    const int full = p.top_k * p.steps;
    row = -1;
    while (place < end) {
      int f0;
      const int r = p.by_row.divmod(place, f0), f1 = min(full, f0 + end - place);
      place += p.row_places - f0;
      if (f0 >= full) continue;
      int h;
      const int t = p.heads.divmod(r, h);
      // the window of a full list is read along with the row's request
      from = f0 + (f1 - f0) * member / p.team;
      const int first = p.by_steps.div(from);
      const int ahead = first + lane < p.top_k ? __ldg(p.blocks + int64_t(r) * p.top_k + first + lane) : -1;
      const int b = __ldg(p.batch_indices + t);
      pos = __ldg(p.positions + t);
      if (b < 0) continue;  // a row without a token: nothing is written
      int n = 0;
      bool bad = b >= p.batch || pos < 0;
      if (!bad) {
        start = __ldg(p.kv_indptr + b);
        n = p.page_size.div(pos) + 1;
        bad = n > __ldg(p.kv_indptr + b + 1) - start;
      }
      if (bad) {
        if (lane == 0 && member == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
        n = 0;
      }
      to = f0 + (f1 - f0) * (member + 1) / p.team;
      if (n < p.top_k) {
        const int a = int(int64_t(f0) * n / p.top_k), b1 = int(int64_t(f1) * n / p.top_k);
        from = a + (b1 - a) * member / p.team;
        to = a + (b1 - a) * (member + 1) / p.team;
      }
      at = p.by_steps.div(from);
      row = r;
      fresh = true;
      window(at == first, ahead);
      return;
    }
  }
  // The next 32 entries; `ahead` holds them where `known`.
  __device__ __forceinline__ void window(bool known = false, int ahead = -1) {
    page = -1;
    begin = end_slot = 0;
    const int e = at + lane;
    if (e * p.steps < to) {
      const int block = known ? ahead : __ldg(p.blocks + int64_t(row) * p.top_k + e);
      if (block >= 0) {
        const int seen = p.page_size.div(pos) + 1;
        if (block < seen) {
          page = __ldg(p.kv_indices + start + block);
          begin = max(0, from - e * p.steps) * kTile;
          end_slot = min(block < seen - 1 ? int(p.page_size.d) : pos - block * int(p.page_size.d) + 1,
                         p.steps > 1 ? (to - e * p.steps) * kTile : int(p.page_size.d));
        }
        if (page < 0 || page >= p.num_pages) {
          record_error(p.st, BSKV_ERR_DEVICE_INDEX);
          end_slot = 0;
        }
      }
    }
    at += 32;
    todo = __ballot_sync(0xffffffffu, begin < end_slot);
  }
  // Moves to an entry that has tokens left; false: the piece has none.
  __device__ __forceinline__ bool seek() {
    if (entry >= 0) return true;
    while (!todo && at * p.steps < to) window();
    if (!todo) return false;
    entry = __ffs(todo) - 1;
    todo &= todo - 1;
    slot = __shfl_sync(0xffffffffu, begin, entry);
    return true;
  }
};

// A stage holds, for each 64-column half, what one copy brings of a page: its rows of K, then its rows of V, 128
// bytes each with the 128-byte swizzle. So the second eight rows are `eight` bytes behind the first: 1024, or 2048
// with pages of eight, of which a tile takes two.
__device__ __forceinline__ uint32_t tile_row(uint32_t base, int r, int hf, uint32_t eight) {
  return base + hf * (2 * kPanel) + (r >> 3) * eight + (r & 7) * 128;
}

// Two weights as sums of two 16-bit values each: what the first leaves of them, half a step of theirs at most, is
// held by the second to half a step of its own.
template <typename T>
__device__ __forceinline__ void two_parts(float a, float b, uint32_t& first, uint32_t& second) {
  first = MmaOp<T>::pack(a, b);
  float2 f;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    f = make_float2(__uint_as_float(first << 16), __uint_as_float(first & 0xffff0000u));
  else
    f = __half22float2(*reinterpret_cast<const __half2*>(&first));
  second = MmaOp<T>::pack(a - f.x, b - f.y);
}

// A pair of values with the greatest number of their sign in place of infinities (and some number of NaN).
template <typename T>
__device__ __forceinline__ uint32_t finite_values(uint32_t x) {
  uint32_t y;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7f7f7f7fu));
  else
    asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7bff7bffu));
  return y;
}

// One tile of 16 tokens for the query heads of a row: up to eight, or WIDE up to 16. v0 and v1 of the two groups of
// eight tokens are attended to. With up to eight heads o[n][2] and o[n][3], the accumulators of rows 8 to 15, belong to
// the weights' second parts.
template <typename T, int D, bool WIDE>
__device__ __forceinline__ void attend_tile(uint32_t k_at, uint32_t v_at, uint32_t eight, int v0, int v1, float scale_log2, int lane,
                                            const uint32_t (&qa)[D / 16][4], float (&o)[D / 8][4], float& m0,
                                            float& m1, float& l0, float& l1) {
  using Mma = MmaOp<T>;
  const int cq = lane & 3;
  if (v0 + v1 < kTile) {
    // slots that are not attended to may hold anything: 0 * NaN must not reach the output
    for (int i = lane; i < kTile * (D / 8); i += 32) {
      const int r = i / (D / 8), c = i % (D / 8);
      if ((r & 7) >= (r < 8 ? v0 : v1)) sts128(tile_row(v_at, r, c >> 3, eight) + (c & 7) * 16, make_uint4(0, 0, 0, 0));
    }
    __syncwarp();
  }
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  {
    const int mi = lane >> 3, r = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int dim = kk * 16 + (mi & 1) * 8;
      uint32_t b0, b1, b2, b3;
      ldsm_x4(tile_row(k_at, r, dim / 64, eight) + ((((dim % 64) / 8) ^ (r & 7)) << 4), b0, b1, b2, b3);
      Mma::run(s[0], qa[kk], b0, b1);
      Mma::run(s[1], qa[kk], b2, b3);
    }
  }
  // m0 and m1 are the references that weights are relative to: the greatest logit, less 15 in fp16. So these weights go up
  // to 2^15, and one is lost below 2^-39 of the greatest, not below 2^-24 (many of which can be much of the sum).
  constexpr float kBelow = std::is_same<T, __half>::value ? 15.f : 0.f;
  float mx0 = -FLT_MAX, mx1 = -FLT_MAX;  // finite: a logit of -inf has no weight, in a tile of only such ones too
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int valid = nt ? v1 : v0;
#pragma unroll
    for (int e = 0; e < (WIDE ? 4 : 2); ++e) s[nt][e] = 2 * cq + (e & 1) < valid ? s[nt][e] * scale_log2 : -INFINITY;
    mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
    if constexpr (WIDE) mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
  }
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
  const float mn0 = fmaxf(m0, mx0 - kBelow), a0 = fast_exp2(m0 - mn0);
  m0 = mn0;
  float mn1 = 0.f, a1 = a0;
  if constexpr (WIDE) {
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    mn1 = fmaxf(m1, mx1 - kBelow);
    a1 = fast_exp2(m1 - mn1);
    m1 = mn1;
  }
  float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    s[nt][0] = fast_exp2(s[nt][0] - mn0);
    s[nt][1] = fast_exp2(s[nt][1] - mn0);
    ps0 += s[nt][0] + s[nt][1];
    if constexpr (WIDE) {
      s[nt][2] = fast_exp2(s[nt][2] - mn1);
      s[nt][3] = fast_exp2(s[nt][3] - mn1);
      ps1 += s[nt][2] + s[nt][3];
    }
  }
  l0 = l0 * a0 + ps0;
  if constexpr (WIDE) l1 = l1 * a1 + ps1;
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    o[n][0] *= a0;
    o[n][1] *= a0;
    o[n][2] *= a1;
    o[n][3] *= a1;
  }
  // The product with V takes weights of 16 bits. Rounded to those they made the output's error against 64 bits a quarter
  // larger than its own rounding does (bf16: 2.1e-3 of its norm, so 1.65e-3); in two parts they add nothing to be seen.
  // Times are the same for up to eight heads (64 requests of 8 x 4 heads 47.9 and 47.7 us), for 16 heads 49.5 and 50.9
  // with 128 dims, 66.5 and 70.0 with 64.
  uint32_t pa[4], pb[4];
  two_parts<T>(s[0][0], s[0][1], pa[0], pb[0]);
  two_parts<T>(s[1][0], s[1][1], pa[2], pb[2]);
  if constexpr (WIDE) {
    two_parts<T>(s[0][2], s[0][3], pa[1], pb[1]);
    two_parts<T>(s[1][2], s[1][3], pa[3], pb[3]);
  } else {
    pa[1] = pb[0];
    pa[3] = pb[2];
  }
  {
    const int mi = lane >> 3, r = (mi & 1) * 8 + (lane & 7);
#pragma unroll
    for (int dd = 0; dd < D / 16; ++dd) {
      const int dim = dd * 16 + (mi >> 1) * 8;
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(tile_row(v_at, r, dim / 64, eight) + ((((dim % 64) / 8) ^ (r & 7)) << 4), b0, b1, b2, b3);
      Mma::run(o[2 * dd], pa, b0, b1);
      Mma::run(o[2 * dd + 1], pa, b2, b3);
      // a second part may be zero or negative: times infinity it must not meet the first's product
      if constexpr (WIDE) {
        Mma::run(o[2 * dd], pb, finite_values<T>(b0), finite_values<T>(b1));
        Mma::run(o[2 * dd + 1], pb, finite_values<T>(b2), finite_values<T>(b3));
      }
    }
  }
}

// States in shared memory: query head g of warp w has D values at (w * group + g) * D, value d at d ^ 4 (g % 8), so
// that neither the fragments' stores nor the joining threads' loads meet in a bank more than twice.
__device__ __forceinline__ int state_at(int row, int g, int d, int D) { return row * D + (d ^ ((g & 7) << 2)); }

template <typename T, int D, bool WIDE, int STAGES>
__global__ void __launch_bounds__(kWarps * 32, 1)
    decode_blocks_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ BlocksParams p) {
  using R = Ring<D, STAGES>;
  using Mma = MmaOp<T>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float top[kWarps][16], sum[kWarps][16];  // of each warp's state
  __shared__ int finished[kWarps];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem + warp * R::kBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * R::kBytes) + warp * STAGES;
  StageInfo* infos = reinterpret_cast<StageInfo*>(smem + kWarps * R::kBytes + kWarps * STAGES * 8) + warp * STAGES;
  float* states = reinterpret_cast<float*>(smem + kWarps * R::kBytes + kWarps * STAGES * (8 + 16));
  const int team = warp / p.team, member = warp - team * p.team, first_warp = warp - member, threads = p.team * 32;
  const int worker = team * gridDim.x + blockIdx.x;  // every SM has one team before any has two
  if (worker >= p.workers) return;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    prefetch_tensormap(&kv_map);
  }
  __syncwarp();
  const bool forced = forced_timeout(p.st);
  const uint64_t policy = l2_evict_first_policy();
  const int ps = int(p.page_size.d);
  const uint32_t eight = ps < kTile ? kPanel : kPanel / 2, v_at = ps < kTile ? kPanel / 2 : kPanel;

  // Copies the next tile of the walk into a stage; a piece without tokens is a tile of none.
  Walk walk(p, worker, member, lane);
  uint32_t issued = 0;
  auto issue = [&]() {
    if (!walk.live()) return;
    const int stage = issued % STAGES;
    uint8_t* to = ring + stage * R::kStageBytes;
    StageInfo info{walk.row, 0, walk.fresh ? kFirst : 0};
    walk.fresh = false;
    int h;
    p.heads.divmod(walk.row, h);
    if (!walk.seek()) {
      if (lane == 0) mbar_arrive(&bars[stage]);
    } else if (ps >= kTile) {
      const int page = __shfl_sync(0xffffffffu, walk.page, walk.entry), end = __shfl_sync(0xffffffffu, walk.end_slot, walk.entry);
      const int slot = walk.slot, left = end - slot;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[stage], uint32_t(R::kStageBytes));
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
          tma_load_5d_hint(to + hf * 2 * kPanel, &kv_map, hf * 64, slot, h, 0, page, &bars[stage], policy);
      }
      info.valid = min(left, 8) | max(0, min(left - 8, 8)) << 16;
      walk.slot += kTile;
      if (walk.slot >= end) walk.entry = -1;
    } else {  // two pages of eight
      const int page0 = __shfl_sync(0xffffffffu, walk.page, walk.entry), c0 = __shfl_sync(0xffffffffu, walk.end_slot, walk.entry);
      walk.entry = -1;
      int page1 = -1, c1 = 0;
      if (walk.seek()) {
        page1 = __shfl_sync(0xffffffffu, walk.page, walk.entry);
        c1 = __shfl_sync(0xffffffffu, walk.end_slot, walk.entry);
        walk.entry = -1;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[stage], uint32_t(c1 ? R::kStageBytes : R::kStageBytes / 2));
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          tma_load_5d_hint(to + hf * 2 * kPanel, &kv_map, hf * 64, 0, h, 0, page0, &bars[stage], policy);
          if (c1) tma_load_5d_hint(to + hf * 2 * kPanel + kPanel, &kv_map, hf * 64, 0, h, 0, page1, &bars[stage], policy);
        }
      }
      info.valid = c0 | c1 << 16;
    }
    if (!walk.seek()) {
      info.flags |= kLast;
      walk.open();
    }
    if (lane == 0) infos[stage] = info;
    ++issued;
  };
  for (int s = 0; s < STAGES; ++s) issue();
  __syncwarp();

  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const int r0 = lane >> 2, r1 = r0 + 8, cq = lane & 3;
  uint32_t consumed = 0;
  bool ok = true;
  // Every warp of the team goes through the same rows, so they meet at the end of each.
  while (consumed < issued) {
    const int stage = consumed % STAGES;
    const StageInfo info = infos[stage];
    int h;
    const int t = p.heads.divmod(info.row, h);
    if (info.flags & kFirst) {
      const T* q = static_cast<const T*>(p.q) + t * p.q_s0 + int64_t(h) * p.group * p.q_s1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int d = kk * 16 + 2 * cq;
        qa[kk][0] = r0 < p.group ? __ldg(reinterpret_cast<const uint32_t*>(q + r0 * p.q_s1 + d)) : 0u;
        qa[kk][1] = WIDE && r1 < p.group ? __ldg(reinterpret_cast<const uint32_t*>(q + r1 * p.q_s1 + d)) : 0u;
        qa[kk][2] = r0 < p.group ? __ldg(reinterpret_cast<const uint32_t*>(q + r0 * p.q_s1 + d + 8)) : 0u;
        qa[kk][3] = WIDE && r1 < p.group ? __ldg(reinterpret_cast<const uint32_t*>(q + r1 * p.q_s1 + d + 8)) : 0u;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    if (ok) ok = warp_wait(&bars[stage], (consumed / STAGES) & 1u, p.st, forced);
    if (ok) {
      const uint32_t at = smem_u32(ring + stage * R::kStageBytes);
      if (info.valid)
        attend_tile<T, D, WIDE>(at, at + v_at, eight, info.valid & 0xffff, info.valid >> 16, p.scale_log2, lane, qa, o,
                                m0, m1, l0, l1);
      ++consumed;
      __syncwarp();
      if (lane == 0) fence_proxy_async_smem();
      issue();
      __syncwarp();
    }
    if (ok && !(info.flags & kLast)) continue;

    // this warp's state, relative to its own reference
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    if constexpr (WIDE) {
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    } else {
      // a second part may be zero or negative: an infinite value counts by the first alone
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        if (fabsf(o[n][0]) < INFINITY) o[n][0] += o[n][2];
        if (fabsf(o[n][1]) < INFINITY) o[n][1] += o[n][3];
      }
    }
    if (r0 < p.group) {
      if (cq == 0) {
        top[warp][r0] = m0;
        sum[warp][r0] = l0;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(states + state_at(warp * p.group + r0, r0, n * 8 + 2 * cq, D)) = make_float2(o[n][0], o[n][1]);
    }
    if (WIDE && r1 < p.group) {
      if (cq == 0) {
        top[warp][r1] = m1;
        sum[warp][r1] = l1;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(states + state_at(warp * p.group + r1, r1, n * 8 + 2 * cq, D)) = make_float2(o[n][2], o[n][3]);
    }
    // a warp whose wait gave up comes here too, wherever it was, and all leave together
    if (!bar_and(1 + team, threads, ok)) {
      ok = false;
      break;
    }
    const Pieces pieces = pieces_of(p, info.row);
    const int count = pieces.last - pieces.first + 1;
    T* out = static_cast<T*>(p.out) + t * p.o_s0 + int64_t(h) * p.group * p.o_s1;
    float* lse = p.lse ? p.lse + int64_t(t) * p.num_qo_heads + h * p.group : nullptr;
    // a row's slots follow one another: teams before it and rows before it have had one each
    const int64_t slot0 = pieces.first + info.row;
    const int64_t base = (slot0 + (worker - pieces.first)) * p.group;
    for (int i = tid - 32 * first_warp; i < p.group * (D / 4); i += threads) {
      const int g = i / (D / 4), d = i % (D / 4) * 4;
      float m = -INFINITY, total = 0.f;
      for (int w = first_warp; w < first_warp + p.team; ++w) m = fmaxf(m, top[w][g]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = first_warp; w < first_warp + p.team; ++w) {
        const float l = sum[w][g];
        if (l == 0.f) continue;  // no token
        const float f = fast_exp2(top[w][g] - m);
        const float4 x = *reinterpret_cast<const float4*>(states + state_at(w * p.group + g, g, d, D));
        total = fmaf(f, l, total);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const float z = total == 0.f ? -INFINITY : (m + __log2f(total)) * kLn2;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (count == 1) {
        *reinterpret_cast<uint2*>(out + g * p.o_s1 + d) = make_uint2(Mma::pack(acc.x, acc.y), Mma::pack(acc.z, acc.w));
        if (lse && d == 0) lse[g] = z;
      } else {
        *reinterpret_cast<float4*>(p.ws_o + (base + g) * D + d) = acc;
        if (d == 0) p.ws_lse[base + g] = z;
      }
    }
    bar_and(1 + team, threads, true);  // the states are read, what was written is ordered before the count
    if (count == 1) continue;
    if (member == 0 && lane == 0) finished[team] = atomic_add_acq_rel(p.counters + info.row, 1);
    bar_and(1 + team, threads, true);
    if (finished[team] != count - 1) continue;
    // the row's last piece: joins the states of all of them, in their order; those without a token (lse
    // -inf) are passed over
    for (int i = tid - 32 * first_warp; i < p.group * (D / 4); i += threads) {
      const int g = i / (D / 4), d = i % (D / 4) * 4;
      constexpr int kAhead = 4;
      float m = -INFINITY, total = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c0 = 0; c0 < count; c0 += kAhead) {
        float z[kAhead];
        float4 x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          z[j] = -INFINITY;
          if (c0 + j < count) {
            const int64_t from = (slot0 + c0 + j) * p.group + g;
            z[j] = __ldcg(p.ws_lse + from);
            x[j] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + from * D + d));
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (z[j] == -INFINITY) continue;
          const float mn = fmaxf(m, z[j]);
          const float sc = m == -INFINITY ? 0.f : expf(m - mn), f = expf(z[j] - mn);
          total = total * sc + f;
          acc.x = acc.x * sc + f * x[j].x;
          acc.y = acc.y * sc + f * x[j].y;
          acc.z = acc.z * sc + f * x[j].z;
          acc.w = acc.w * sc + f * x[j].w;
          m = mn;
        }
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      *reinterpret_cast<uint2*>(out + g * p.o_s1 + d) = make_uint2(Mma::pack(acc.x * inv, acc.y * inv), Mma::pack(acc.z * inv, acc.w * inv));
      if (lse && d == 0) lse[g] = total == 0.f ? -INFINITY : m + logf(total);
    }
    if (member == 0 && lane == 0) p.counters[info.row] = 0;  // ready for the next run
  }
  if (!ok) {
    // the copies in flight land before the warp leaves (bounded, not forcible)
    for (uint32_t s = consumed; s < issued; ++s) mbar_wait(&bars[s % STAGES], (s / STAGES) & 1u, p.st, false);
  }
}

template <typename T, int D, bool WIDE, int STAGES>
bskv_status launch(const CUtensorMap& map, const BlocksParams& p, int grid, cudaStream_t st) {
  using R = Ring<D, STAGES>;
  auto kern = decode_blocks_kernel<T, D, WIDE, STAGES>;
  static_assert(sizeof(StageInfo) <= 16, "stage infos");
  const size_t smem = 1024 + kWarps * (R::kBytes + STAGES * (8 + 16)) + size_t(kWarps) * p.group * D * 4;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "run_decode_blocks: cudaFuncSetAttribute")) return s;
  kern<<<unsigned(grid), kWarps * 32, smem, st>>>(map, p);
  return cuda_check(cudaGetLastError(), "run_decode_blocks launch");
}

// Stages by what shared memory holds beside the warps' states: with more than eight query heads of 128
// dims these take 64 KB.
template <typename T>
bskv_status launch_any(const CUtensorMap& map, const BlocksParams& p, int D, int grid, cudaStream_t st) {
  if (p.group <= 8) return D == 64 ? launch<T, 64, false, 5>(map, p, grid, st) : launch<T, 128, false, 3>(map, p, grid, st);
  return D == 64 ? launch<T, 64, true, 5>(map, p, grid, st) : launch<T, 128, true, 2>(map, p, grid, st);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

BlocksWorkspace blocks_workspace(const bskv_plan* plan) {
  BlocksWorkspace w{};
  const size_t rows = size_t(plan->M) * size_t(plan->num_kv_heads), blocks = (size_t(plan->max_blocks) + 3) & ~size_t(3);
  const size_t group = size_t(plan->num_qo_heads / std::max(1, plan->num_kv_heads));
  const size_t slots = rows + size_t(plan->workers);
  w.stride = int(blocks);
  size_t at = 0;
  const size_t heads = size_t(std::max(1, plan->num_kv_heads)), query = heads * blocks * 4;
  w.slice = int64_t(std::min(std::max<size_t>(1, kSelectBytes / query), size_t(kSelectSlice)));
  w.scores = at; at += align256(std::min(rows, size_t(w.slice) * heads) * blocks * 4);
  w.states = at; at += align256(slots * group * size_t(plan->head_dim) * 4);
  w.lse = at; at += align256(slots * group * 4);
  w.total = at;
  return w;
}

bskv_status check_blocks_run(const char* who, const bskv_plan* plan, const int32_t* batch_indices,
                             const int32_t* positions, const int32_t* kv_indptr, const int32_t* kv_indices,
                             int32_t batch, const int32_t* blocks, const void* float_ws, size_t float_ws_bytes) {
  if (!plan || plan->kind != KIND_BLOCKS) { set_error("%s: not a block-sparse decode plan", who); return BSKV_ERR_INVALID_ARG; }
  if (!plan->meta_dev) { set_error("%s: plan not uploaded (bskv_plan_upload)", who); return BSKV_ERR_INVALID_ARG; }
  if (batch < 0) { set_error("%s: batch=%d", who, batch); return BSKV_ERR_INVALID_ARG; }
  if (plan->M == 0) return BSKV_OK;
  if (!batch_indices || !positions || !kv_indptr || !kv_indices || !blocks) { set_error("%s: NULL argument", who); return BSKV_ERR_INVALID_ARG; }
  if ((reinterpret_cast<uintptr_t>(batch_indices) | reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(kv_indptr) |
       reinterpret_cast<uintptr_t>(kv_indices) | reinterpret_cast<uintptr_t>(blocks)) & 3) {
    set_error("%s: index arrays must be 4-byte aligned", who);
    return BSKV_ERR_INVALID_ARG;
  }
  if (!float_ws || float_ws_bytes < plan->float_ws_bytes) {
    set_error("%s: float workspace of %zu bytes, %zu needed", who, float_ws_bytes, plan->float_ws_bytes);
    return BSKV_ERR_WORKSPACE_TOO_SMALL;
  }
  if (!aligned16(float_ws)) { set_error("%s: the float workspace must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  return BSKV_OK;
}

}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_run_decode_blocks(
    const bskv_plan* plan, const void* q, const int64_t* q_strides, const void* kv_cache,
    const int64_t* kv_strides, const int32_t* blocks, const int32_t* batch_indices,
    const int32_t* positions, const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch,
    void* out, const int64_t* out_strides, float* lse, float sm_scale, void* float_ws,
    size_t float_ws_bytes, void* stream) {
  BSKV_NVTX_RANGE("bskv_run_decode_blocks");
  const char* who = "run_decode_blocks";
  if (bskv_status s = check_blocks_run(who, plan, batch_indices, positions, kv_indptr, kv_indices, batch, blocks, float_ws, float_ws_bytes)) return s;
  if (plan->M == 0) return BSKV_OK;
  if (!q || !q_strides || !out || !out_strides || !kv_cache || !kv_strides) { set_error("%s: NULL argument", who); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) { set_error("%s: tensors must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 4; ++i)
    if (kv_strides[i] <= 0 || kv_strides[i] % 8) {
      set_error("%s: kv stride %d (%lld elements) must be positive and 16-byte aligned", who, i, (long long)kv_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] < 0 || q_strides[i] % 8 || out_strides[i] < 0 || out_strides[i] % 8) {
      set_error("%s: q and out strides must be multiples of 16 bytes", who);
      return BSKV_ERR_INVALID_ARG;
    }
  if (plan->num_pages == 0) { set_error("%s: a cache without pages", who); return BSKV_ERR_INVALID_ARG; }
  const BlocksWorkspace ws = blocks_workspace(plan);
  uint8_t* base = static_cast<uint8_t*>(float_ws);
  BlocksParams p{};
  p.q = q; p.q_s0 = q_strides[0]; p.q_s1 = q_strides[1];
  p.out = out; p.o_s0 = out_strides[0]; p.o_s1 = out_strides[1];
  p.lse = lse;
  p.blocks = blocks; p.batch_indices = batch_indices; p.positions = positions; p.kv_indptr = kv_indptr; p.kv_indices = kv_indices;
  p.ws_o = reinterpret_cast<float*>(base + ws.states); p.ws_lse = reinterpret_cast<float*>(base + ws.lse);
  p.num_rows = plan->M * plan->num_kv_heads;
  p.counters = plan->counters_dev + p.num_rows;  // behind the selection's
  p.top_k = plan->top_k; p.team = plan->team; p.workers = plan->workers; p.per_worker = plan->per_worker;
  p.steps = plan->steps; p.row_places = plan->row_places; p.places = p.num_rows * plan->row_places;
  p.group = plan->num_qo_heads / plan->num_kv_heads; p.num_qo_heads = plan->num_qo_heads;
  p.batch = batch; p.num_pages = plan->num_pages;
  p.heads = FastDiv(plan->num_kv_heads); p.page_size = FastDiv(plan->page_size);
  p.by_row = FastDiv(plan->row_places); p.by_worker = FastDiv(plan->per_worker); p.by_steps = FastDiv(plan->steps);
  p.scale_log2 = sm_scale_log2(sm_scale, plan->head_dim);
  if (bskv_status s = status_args(&p.st)) return s;
  const int ps = plan->page_size, D = plan->head_dim;
  const uint64_t dims[5] = {uint64_t(D), uint64_t(ps), uint64_t(plan->num_kv_heads), 2, uint64_t(plan->num_pages)};
  const uint64_t strides[4] = {uint64_t(kv_strides[3]) * 2, uint64_t(kv_strides[2]) * 2, uint64_t(kv_strides[1]) * 2,
                               uint64_t(kv_strides[0]) * 2};
  const uint32_t box[5] = {64, uint32_t(std::min(ps, kTile)), 1, 2, 1};  // K and V of a page
  CUtensorMap map;
  if (bskv_status s = encode_tiled(&map, plan->dtype == BSKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                   5, kv_cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = std::min(plan->num_sms, plan->workers);
  return plan->dtype == BSKV_BF16 ? launch_any<__nv_bfloat16>(map, p, D, grid, st) : launch_any<__half>(map, p, D, grid, st);
}
