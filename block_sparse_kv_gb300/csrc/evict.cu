// Eviction from a paged cache by accumulated attention weight: which tokens stay, and the
// compaction of their rows.
//
// Selection. Per (request, kv head): the first `sink` and the last `recent` tokens stay, and of
// the others the k of highest score (NaN above everything, -0 = +0, the lowest slot among equals).
// Scores become 32-bit keys of the same order; three histogram passes (11, 11 and 10 bits) find
// the k-th largest key T, and one pass in slot order keeps the keys above T and the first ones
// equal to it. Counts are integers, so the result does not depend on the order of the atomics.
// The scores are read once, into shared memory; what bounds the kernel is latency: about 6000
// cycles for three dependent reads (request, page, scores) and 1500 per pass. So few long requests
// are shared by a cluster of up to 8 CTAs: 131072 tokens of 8 heads took 340 us on one CTA per head
// and 21 us so. With as many rows as SMs a cluster only adds its barriers (8192 tokens, 128 rows:
// the operator 36.6 us, in clusters of two 44.9). CTAs have 256 threads where a share is at most
// 2048 tokens, else 1024 (512 rows of 1088 tokens: 100 against 114 us; 8192 tokens: 40.8 against
// 36.5).
//
// Compaction. Kept tokens move to the front in their order: row j comes from slot kept[j] >= j.
// Within one cache it is done in place: rows are taken in waves of ascending j, every read of a
// wave before its first write (one barrier), and a later wave only reads slots above every slot
// written so far, which is why it may be read before that. A wave's rows therefore never meet, so
// K, V, the scores and the 4-bit scales each go through their waves on their own CTA, or, where
// there are few requests, on a cluster of up to 8 that shares the waves (131072 tokens of 8 heads
// halved: 178 us; 8 requests of 8192 tokens halved: 150 us on one CTA each, 67 us on 4). The
// cluster's barrier waits for what its threads wrote and read before, so it pays to hold many rows
// between two: 16 a thread, where 8 with the next 8 under way took 244 and 83 us. Into other pages
// there is nothing to order and blocks of rows have CTAs too.
// Bound by memory: of the widths 64, 128 and 256 bytes per row and CTA, whole rows were fastest in
// place (138, 115 and 104 us), and eight CTAs per SM with two rows a thread ahead of four with
// four (104 and 113 us). 537 MB in place in 83 us: 6.4 TB/s.
#include <algorithm>

#include "cache_common.cuh"
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
  FastDiv page_size;
  int off_req, off_src, off_src_ptr, off_dst;
  int sink, recent, in_place;
  int held;            // selection: groups of four keys of a CTA that shared memory holds
  int planes;          // compaction: column slices
};

// {tokens, kept tokens, first of them in `kept`, first destination page entry}
__device__ __forceinline__ int4 request_of(const EvictParams& p, int b) {
  return __ldg(reinterpret_cast<const int4*>(p.meta + p.off_req) + b);
}

// ---------------------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------------------

constexpr int kBins = 2048;
constexpr int kSelectFours = 8192;  // most groups of four keys that a CTA's shared memory holds; more are read again
constexpr int kMaxCluster = 8;      // the portable size
constexpr int kClusterTokens = 2048;  // least tokens of a CTA of a cluster

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes +0
  if (x != x) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the threads below of one value per thread; the sums go through warp_sums[32].
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int s = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
  return s + x - v;
}

// One (request, kv head) per cluster of `ctas` CTAs, each with a contiguous part of the tokens, four
// of a page to a thread at a time. Protected tokens among them get the key 0, below every score's.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const __grid_constant__ EvictParams p, int ctas) {
  constexpr int kWarps = THREADS / 32, kPer = kBins / THREADS;  // bins per thread
  extern __shared__ uint4 keys[];
  const bool cluster = THREADS >= kBins / 2 && ctas > 1;  // a bin of a cluster CTA's share per thread
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ int sums[kBins / 2], totals[kMaxCluster];  // a cluster's bins: this CTA's share, each share's total
  __shared__ int warp_sums[32], warp_eq[32];
  __shared__ __align__(8) int counts[2];
  __shared__ uint32_t found_digit;
  __shared__ int found_rest;
  const int b = blockIdx.z, h = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  const int32_t* pages = p.meta + p.off_src + __ldg(p.meta + p.off_src_ptr + b);
  const int4 rq = request_of(p, b);
  const int L = rq.x, K = rq.y;
  int32_t* kept = p.kept + h * p.total + rq.z;
  if (K == L) {
    for (int j = rank * THREADS + tid; j < K; j += ctas * THREADS) kept[j] = j;
    return;
  }
  for (int j = rank * THREADS + tid; j < p.sink; j += ctas * THREADS) kept[j] = j;
  for (int j = rank * THREADS + tid; j < p.recent; j += ctas * THREADS) kept[K - p.recent + j] = L - p.recent + j;
  const int first = p.sink, end = L - p.recent, k = K - p.sink - p.recent;
  if (k == 0) return;
  const int fours = (end - (first & ~3) + 3) >> 2;
  const int share = ((fours + ctas - 1) / ctas + 31) & ~31;
  const int g0 = min(fours, rank * share), n = min(fours, g0 + share) - g0;  // this CTA's groups of four
  const int base = (first & ~3) + 4 * g0;
  const float* scores = p.scores + h * p.w_s1;
  const bool held = n <= p.held;
  auto load = [&](int i) {
    const int t = base + 4 * i;
    int slot;
    const int pg = p.page_size.divmod(t, slot);
    const float4 s = __ldg(reinterpret_cast<const float4*>(scores + __ldg(pages + pg) * p.w_s0 + slot));
    return make_uint4(t >= first && t < end ? order_key(s.x) : 0u, t + 1 >= first && t + 1 < end ? order_key(s.y) : 0u,
                      t + 2 >= first && t + 2 < end ? order_key(s.z) : 0u, t + 3 >= first && t + 3 < end ? order_key(s.w) : 0u);
  };
  if (held) {
#pragma unroll 4
    for (int i = tid; i < n; i += THREADS) keys[i] = load(i);
  }
  auto key = [&](int i) { return held ? keys[i] : load(i); };
  auto all_sync = [&]() {
    __syncwarp();
    if (cluster) cluster_sync();
    else __syncthreads();
  };

  // digits of T from the top; `rest` of the keys that share the digits so far are at or above T
  uint32_t T = 0;
  int rest = k;
  for (int i = tid; i < kBins; i += THREADS) hist[0][i] = 0;
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    int* mine = hist[pass & 1];
    auto count = [&](uint32_t x) {
      if (pass == 0 || (x ^ T) >> (shift + bits) == 0)
        atomicAdd(&mine[(x >> shift) & ((1u << bits) - 1)], 1);
    };
#pragma unroll 2
    for (int i = tid; i < n; i += THREADS) {
      const uint4 x = key(i);
      count(x.x);
      count(x.y);
      count(x.z);
      count(x.w);
    }
    all_sync();
    // thread i's bins are below those of the threads before it: sums over these are of larger keys
    if (cluster) {
      // each CTA adds up its share of the bins over the cluster; the total says whose share has T's digit
      const int bins = kBins / ctas;
      int sum = 0;
      if (tid < bins) {
        const uint32_t from = smem_u32(mine + rank * bins + tid);
        int v[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) v[c] = c < ctas ? ld_cluster_s32(mapa_shared(from, uint32_t(c))) : 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) sum += v[c];
        sums[tid] = sum;
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) warp_sums[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_sums[lane] : 0);
        if (lane < ctas) st_cluster_u32(mapa_shared(smem_u32(&totals[rank]), uint32_t(lane)), uint32_t(sum));
      }
      __syncwarp();
      cluster_sync();
      int owner = ctas - 1;
      for (; owner > 0 && rest > totals[owner]; --owner) rest -= totals[owner];
      const int bin = tid < bins ? ld_cluster_s32(mapa_shared(smem_u32(sums + bins - 1 - tid), uint32_t(owner))) : 0;
      const int before = block_scan<THREADS>(bin, warp_sums);
      if (before < rest && rest <= before + bin) {
        found_digit = uint32_t(owner * bins + bins - 1 - tid);
        found_rest = rest - before;
      }
    } else {
      const int top = kBins - kPer * tid;
      int bin[kPer], sum = 0;
#pragma unroll
      for (int u = 0; u < kPer; ++u) sum += bin[u] = mine[top - kPer + u];
      int before = block_scan<THREADS>(sum, warp_sums);
      if (before < rest && rest <= before + sum) {
#pragma unroll
        for (int u = kPer - 1; u >= 0; --u) {
          if (before < rest && rest <= before + bin[u]) {
            found_digit = uint32_t(top - kPer + u);
            found_rest = rest - before;
          }
          before += bin[u];
        }
      }
    }
    if (pass < 2)  // its readers were done before the barrier that this pass began with
      for (int i = tid; i < kBins; i += THREADS) hist[(pass + 1) & 1][i] = 0;
    __syncthreads();
    T |= found_digit << shift;
    rest = found_rest;
  }

  // each warp takes a contiguous part of the CTA's: counts, then places
  const int part = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int i0 = min(n, warp * part), i1 = min(n, i0 + part);
  int above = 0, equal = 0;
#pragma unroll 2
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint4 x = key(i);
    above += (x.x > T) + (x.y > T) + (x.z > T) + (x.w > T);
    equal += (x.x == T) + (x.y == T) + (x.z == T) + (x.w == T);
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    warp_sums[warp] = above;
    warp_eq[warp] = equal;
  }
  __syncthreads();
  const int wa = lane < kWarps ? warp_sums[lane] : 0, we = lane < kWarps ? warp_eq[lane] : 0;
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
  int eq = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
  if (cluster) {
    if (warp == 0) {
      const int a = __reduce_add_sync(0xffffffffu, wa), e = __reduce_add_sync(0xffffffffu, we);
      if (lane == 0) {
        counts[0] = a;
        counts[1] = e;
      }
    }
    __syncwarp();
    cluster_sync();
    int2 c = make_int2(0, 0);
    if (lane < rank) c = ld_cluster_v2(mapa_shared(smem_u32(counts), uint32_t(lane)));
    at += __reduce_add_sync(0xffffffffu, c.x);
    eq += __reduce_add_sync(0xffffffffu, c.y);
    __syncwarp();
    cluster_arrive();  // waited for at the end: no CTA leaves while its counts are read
  }
  at += first + min(eq, rest);
  const uint32_t below = (1u << lane) - 1;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint4 x4 = i < i1 ? key(i) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
    bool stay[4];
    int rank_eq = eq;  // equal keys in the slots before
    if (__any_sync(0xffffffffu, x[0] == T || x[1] == T || x[2] == T || x[3] == T)) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m = __ballot_sync(0xffffffffu, x[u] == T);
        rank_eq += __popc(m & below);
        eq += __popc(m);
      }
    }
    int to = at;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      stay[u] = x[u] > T || (x[u] == T && rank_eq < rest);
      rank_eq += x[u] == T;
      const uint32_t m = __ballot_sync(0xffffffffu, stay[u]);
      to += __popc(m & below);
      at += __popc(m);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (stay[u]) kept[to++] = base + 4 * i + u;
  }
  if (cluster) {
    __syncwarp();
    cluster_wait();
  }
}

// ---------------------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveTable = 1024;  // rows whose places a CTA looks up at a time
constexpr int kMoveBlock = 256;   // rows per CTA when copying (16384 of 8 heads in 4 bits: 57.4 us, by 128 58.7, by 512 59.6)
constexpr int kMoveShare = 1024;  // least rows of a CTA of a cluster

// One column slice of a paged tensor's rows: 2^shift units per row (16, 4 or 2 bytes each).
struct Plane {
  uint8_t* base;
  int64_t s0, s_head, s_slot;  // bytes
  int unit, shift;
};
constexpr int kMaxPlanes = 10;
struct MoveParams {
  EvictParams e;
  Plane plane[kMaxPlanes];
};

struct Places {
  int64_t from[kMoveTable], to[kMoveTable];  // bytes from the plane's base; to < 0: stays
};

// The table's rows [0, n) in waves of ROWS per thread. Where a wave's barrier is the CTA's (SHARED
// false), the next wave is read before it.
template <typename U, int ROWS, bool SHARED, typename Sync>
__device__ __forceinline__ void move_rows(const Places& at, uint8_t* base, int shift, int n, Sync sync) {
  const int row = threadIdx.x >> shift, per = kMoveThreads >> shift, wave = per * ROWS;
  base += (threadIdx.x & ((1 << shift) - 1)) * sizeof(U);
  auto read = [&](U (&x)[ROWS], int w) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = w + i * per + row;
      if (j < n && at.to[j] >= 0) x[i] = *reinterpret_cast<const U*>(base + at.from[j]);
    }
  };
  auto write = [&](const U (&x)[ROWS], int w) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = w + i * per + row;
      if (j < n && at.to[j] >= 0) *reinterpret_cast<U*>(base + at.to[j]) = x[i];
    }
  };
  U x0[ROWS] = {};
  if constexpr (SHARED) {
    for (int w = 0; w < n; w += wave) {
      read(x0, w);
      sync();  // every read of the wave before its first write
      write(x0, w);
    }
  } else {
    U x1[ROWS] = {};
    read(x0, 0);
    for (int w = 0; w < n; w += 2 * wave) {
      read(x1, w + wave);
      sync();
      write(x0, w);
      if (w + wave >= n) break;
      read(x0, w + 2 * wave);
      sync();
      write(x1, w + wave);
    }
  }
}

// SHARED: a slice's waves are spread over a cluster of `ctas` CTAs, in place.
template <bool SHARED>
__global__ void __launch_bounds__(kMoveThreads, SHARED ? 2 : 8)
    evict_move_kernel(const __grid_constant__ MoveParams mp, int ctas) {
  constexpr int kRows = SHARED ? 16 : 2;
  __shared__ Places at;
  const EvictParams& p = mp.e;
  const int rank = SHARED ? blockIdx.x % ctas : 0;
  const Plane& pl = mp.plane[SHARED ? blockIdx.x / ctas : blockIdx.x % p.planes];
  const int h = blockIdx.y, b = blockIdx.z;
  const int4 rq = request_of(p, b);
  const int K = rq.y;
  // `kept` is read below and pages are written that the selection reads; and what follows this kernel
  // on the stream follows the selection only if every CTA waits for it
  wait_for_prior_grid();
  if (p.in_place && K == rq.x) return;
  const int32_t* kept = p.kept + h * p.total + rq.z;
  const int32_t* src_pages = p.meta + p.off_src + __ldg(p.meta + p.off_src_ptr + b);
  const int32_t* dst_pages = p.meta + p.off_dst + rq.w;
  uint8_t* base = pl.base + h * pl.s_head;
  // CTA `rank` of a cluster has the rows [wave * rank, wave * (rank + 1)) of every wave * ctas
  const int wave = min(kMoveTable, (kMoveThreads >> pl.shift) * kRows), turn = __ffs(wave) - 1;
  const int j0 = SHARED || p.in_place ? 0 : blockIdx.x / p.planes * kMoveBlock;
  const int j1 = SHARED || p.in_place ? K : min(K, j0 + kMoveBlock);
  const int total = SHARED ? (K + wave * ctas - 1) / (wave * ctas) * wave : j1 - j0;  // rows of this CTA
  for (int r0 = 0; r0 < total; r0 += kMoveTable) {
    const int n = min(kMoveTable, total - r0);
    if (r0 > 0) __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
      const int r = r0 + i, j = SHARED ? ((((r >> turn) * ctas + rank) << turn) | (r & (wave - 1))) : j0 + r;
      const int s = j < j1 ? __ldcg(kept + j) : j;
      int64_t from = 0, to = -1;
      if (j < j1 && !(p.in_place && s == j)) {
        int ss, ds;
        const int sn = p.page_size.divmod(s, ss), dn = p.page_size.divmod(j, ds);
        from = __ldg(src_pages + sn) * pl.s0 + ss * pl.s_slot;
        to = __ldg(dst_pages + dn) * pl.s0 + ds * pl.s_slot;
      }
      at.from[i] = from;
      at.to[i] = to;
    }
    __syncthreads();
    auto sync = [&]() {
      if constexpr (SHARED) {
        __syncwarp();
        cluster_sync();
      } else if (p.in_place) {
        __syncthreads();
      }
    };
    if (pl.unit == 16) move_rows<uint4, kRows, SHARED>(at, base, pl.shift, n, sync);
    else if (pl.unit == 4) move_rows<uint32_t, kRows, SHARED>(at, base, pl.shift, n, sync);
    else move_rows<uint16_t, kRows, SHARED>(at, base, pl.shift, n, sync);
  }
}

// Launches kern(params, ctas) with clusters of `ctas` CTAs along x; early: once every CTA of the
// kernel before it on the stream runs.
template <typename P>
cudaError_t launch_clusters(void (*kern)(P, int), dim3 grid, int threads, size_t smem, int ctas, const P& params,
                            bool early, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {unsigned(ctas), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, params, ctas);
}

template <int THREADS>
bskv_status select(const EvictParams& e, const bskv_plan* plan, int ctas, size_t smem, cudaStream_t st) {
  auto kern = evict_select_kernel<THREADS>;
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed, "evict: cudaFuncSetAttribute"))
    return s;
  const dim3 grid(unsigned(ctas), unsigned(plan->num_kv_heads), unsigned(plan->batch));
  return cuda_check(launch_clusters<EvictParams>(kern, grid, THREADS, smem, ctas, e, false, st), "evict select launch");
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
  e.page_size = FastDiv(plan->page_size);
  e.sink = plan->sink; e.recent = plan->recent; e.in_place = plan->in_place;
  if (compact_scores)
    mp.plane[planes++] = Plane{reinterpret_cast<uint8_t*>(scores), 4 * e.w_s0, 4 * e.w_s1, 4, 4, 0};
  const int64_t rows = int64_t(plan->batch) * plan->num_kv_heads;
  int ctas = 1;
  while (ctas < kMaxCluster && plan->longest / (2 * ctas) >= kClusterTokens && rows * ctas * 2 <= plan->num_sms) ctas *= 2;
  const int share = (((plan->longest + 3) / 4 + ctas) / ctas + 31) & ~31;  // groups of four per CTA, at most
  e.held = std::min(kSelectFours, share);
  const size_t smem = sizeof(uint4) * size_t(e.held);
  const bool big = ctas > 1 || share > 512;
  if (bskv_status s = big ? select<1024>(e, plan, ctas, smem, st) : select<256>(e, plan, ctas, smem, st)) return s;
  e.planes = planes;
  ctas = 1;
  while (plan->in_place && ctas < kMaxCluster && plan->most / (2 * ctas) >= kMoveShare && rows * planes * ctas <= int64_t(4) * plan->num_sms)
    ctas *= 2;
  const int parts = plan->in_place ? ctas : (plan->most + kMoveBlock - 1) / kMoveBlock;
  const dim3 grid(unsigned(planes * parts), unsigned(plan->num_kv_heads), unsigned(plan->batch));
  auto kern = ctas > 1 ? evict_move_kernel<true> : evict_move_kernel<false>;
  return cuda_check(launch_clusters<MoveParams>(kern, grid, kMoveThreads, 0, ctas, mp, true, st), "evict move launch");
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
  // whole rows, or 64 bytes of them where few long requests would leave SMs idle (131072 tokens of one
  // head halved: 61 us, by whole rows 160)
  const bool narrow = plan->in_place && plan->most >= 2 * kMoveShare &&
                      int64_t(plan->batch) * plan->num_kv_heads * plan->head_dim / 16 <= plan->num_sms / kMaxCluster;
  const int cols = narrow ? 64 : 2 * plan->head_dim;
  for (int which = 0; which < 2; ++which)
    for (int col = 0; col < 2 * plan->head_dim; col += cols)
      mp.plane[planes++] = Plane{static_cast<uint8_t*>(kv_cache) + 2 * which * kv_strides[1] + col, 2 * kv_strides[0],
                                 2 * kv_strides[2], 2 * kv_strides[3], 16, narrow ? 2 : plan->head_dim == 128 ? 4 : 3};
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
                               codes_strides[2], codes_strides[3], 16, plan->head_dim == 128 ? 2 : 1};
    mp.plane[planes++] = Plane{static_cast<uint8_t*>(kv_scales) + which * scales_strides[1],
                               scales_strides[0], scales_strides[2], blocks, blocks, 0};
  }
  return run(who, plan, scores, scores_strides, kept, compact_scores != 0, mp, planes,
             static_cast<cudaStream_t>(stream));
}
