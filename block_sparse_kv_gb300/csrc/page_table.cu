// Page table and token map of a batch, made on the GPU from the requests' lengths.
//
// Mathematics. Request b holds len_b tokens, the last new_b of them new:
//   pages_b = ceil(len_b / page_size), fresh_b = pages_b - ceil((len_b - new_b) / page_size),
// and the compressed arrays are exclusive sums of pages_b (kv_indptr) and new_b (qo_indptr). Fresh
// pages come from the end of the free list, request by request, so their places are the exclusive sum
// of fresh_b: every output can be computed on its own once the three sums are known.
//
// Bound by latency (a decode step writes some kilobytes), for prompts by the stores. So there is one
// launch: every CTA makes the sums of the whole batch for itself in shared memory (8 bytes a request
// out of L2; no CTA waits for another) and then writes its share of the page entries and the token
// rows, finding an entry's request by bisection of the sums. A thread writes four rows at a time, one
// 16-byte store each for requests and positions. 64 requests with a new token each: 5.0 us; a million new tokens of
// 256 requests: 8.2 us.
#include <algorithm>

#include "cache_common.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = 8192;  // five numbers per request in shared memory: 160 KB

struct PageTableParams {
  const int32_t *lens, *news;
  int32_t* table;
  int64_t t_s;
  int batch, max_pages, num_pages;
  FastDiv page_size;
  const int32_t *free_pages, *free_count;
  int max_free;
  int32_t* free_left;
  int32_t *kv_indptr, *kv_indices, *kv_last_page_len, *qo_indptr;
  int32_t *batch_indices, *positions;
  int64_t* slots;
  int max_tokens;
  StatusArgs st;
};

struct Lens {
  int len, fresh_from, pages, fresh;  // new tokens: len - first_new
  int first_new;
};

// A request's lengths; one that is negative, or does not fit, counts as empty.
__device__ __forceinline__ Lens lens_of(const PageTableParams& p, int b, bool& bad) {
  Lens r;
  const int len = __ldg(p.lens + b), nw = p.news ? __ldg(p.news + b) : min(len, 1);
  bad = len < 0 || nw < 0 || nw > len || len > p.max_pages * int(p.page_size.d);
  r.len = bad ? 0 : len;
  r.first_new = bad ? 0 : len - nw;
  r.pages = p.page_size.div(r.len + int(p.page_size.d) - 1);
  r.fresh_from = p.free_pages ? p.page_size.div(r.first_new + int(p.page_size.d) - 1) : r.pages;
  r.fresh = r.pages - r.fresh_from;
  return r;
}

// Last i of [0, n) with sums[i] <= x, for ascending sums with sums[0] <= x: the request of entry x.
__device__ __forceinline__ int owner(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_table_kernel(const __grid_constant__ PageTableParams p) {
  extern __shared__ int sums[];  // exclusive sums of pages, new tokens and fresh pages, totals behind
  int* pages = sums;
  int* tokens = pages + p.batch + 1;
  int* fresh = tokens + p.batch + 1;
  int* fresh_from = fresh + p.batch + 1;  // first fresh page, first new token
  int* first_new = fresh_from + p.batch;
  __shared__ int3 warp_sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int free_n = p.free_pages ? __ldg(p.free_count) : 0;
  for (int b = tid; b < p.batch; b += kThreads) {
    bool bad;
    const Lens r = lens_of(p, b, bad);
    if (bad && blockIdx.x == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    pages[b] = r.pages;
    tokens[b] = r.len - r.first_new;
    fresh[b] = r.fresh;
    fresh_from[b] = r.fresh_from;
    first_new[b] = r.first_new;
  }
  if (free_n < 0 || (p.free_pages && free_n > p.max_free)) {
    if (blockIdx.x == 0 && tid == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    free_n = 0;
  }
  __syncthreads();
  // each thread adds up a run of requests, the runs' sums are scanned over the CTA
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  int3 own = make_int3(0, 0, 0);
  for (int b = b0; b < b1; ++b) {
    own.x += pages[b];
    own.y += tokens[b];
    own.z += fresh[b];
  }
  int3 x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, o), c = __shfl_up_sync(0xffffffffu, x.y, o),
              d = __shfl_up_sync(0xffffffffu, x.z, o);
    if (lane >= o) {
      x.x += a;
      x.y += c;
      x.z += d;
    }
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int3 ws = lane < warp ? warp_sums[lane] : make_int3(0, 0, 0);
  x.x += __reduce_add_sync(0xffffffffu, ws.x) - own.x;
  x.y += __reduce_add_sync(0xffffffffu, ws.y) - own.y;
  x.z += __reduce_add_sync(0xffffffffu, ws.z) - own.z;
  for (int b = b0; b < b1; ++b) {
    const int3 v = make_int3(pages[b], tokens[b], fresh[b]);
    pages[b] = x.x;
    tokens[b] = x.y;
    fresh[b] = x.z;
    x.x += v.x;
    x.y += v.y;
    x.z += v.z;
  }
  if (tid == kThreads - 1) {
    pages[p.batch] = x.x;
    tokens[p.batch] = x.y;
    fresh[p.batch] = x.z;
  }
  __syncthreads();
  const int num_entries = pages[p.batch], num_tokens = tokens[p.batch];

  // the id of page j of request b: a fresh one from the free list, else the table's; -1: none
  auto read_id = [&](int b, int j) -> int {
    const int nth = j - fresh_from[b];
    if (nth < 0) return p.table[b * p.t_s + j];
    const int at = free_n - 1 - (fresh[b] + nth);
    return at >= 0 ? __ldg(p.free_pages + at) : -1;
  };
  auto checked = [&](int id) -> int {
    if (id >= 0 && id < p.num_pages) return id;
    record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    return -1;
  };

  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.batch; b += kThreads) {
      p.kv_indptr[b] = pages[b];
      p.qo_indptr[b] = tokens[b];
      if (b < p.batch) {
        const int n = pages[b + 1] - pages[b], len = first_new[b] + tokens[b + 1] - tokens[b];
        p.kv_last_page_len[b] = n > 0 ? len - (n - 1) * int(p.page_size.d) : 0;
      }
    }
    if (tid == 0) {
      if (p.free_left) *p.free_left = max(0, free_n - fresh[p.batch]);
      if (num_tokens > p.max_tokens) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    }
  }
  // rows r0 .. r0 + 3 of the token map
  auto write_rows = [&](int r0) {
    int req[4], pos[4];
    int64_t slot[4];
    int id[4], in_page[4], b = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + i;
      req[i] = pos[i] = -1;
      if (row >= num_tokens || row >= p.max_tokens) continue;
      if (b >= 0 && row >= tokens[b + 1]) b = b + 2 <= p.batch && row < tokens[b + 2] ? b + 1 : -1;  // often the next request's
      if (b < 0) b = owner(tokens, p.batch, row);
      req[i] = b;
      pos[i] = first_new[b] + row - tokens[b];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (req[i] >= 0) id[i] = read_id(req[i], p.page_size.divmod(pos[i], in_page[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      slot[i] = -1;
      if (req[i] >= 0 && (id[i] = checked(id[i])) >= 0) slot[i] = int64_t(id[i]) * p.page_size.d + in_page[i];
    }
    if (r0 + 4 <= p.max_tokens) {
      *reinterpret_cast<int4*>(p.batch_indices + r0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots) {
        *reinterpret_cast<longlong2*>(p.slots + r0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(p.slots + r0 + 2) = make_longlong2(slot[2], slot[3]);
      }
    } else {
      for (int i = 0; r0 + i < p.max_tokens; ++i) {
        p.batch_indices[r0 + i] = i == 0 ? req[0] : i == 1 ? req[1] : req[2];
        p.positions[r0 + i] = i == 0 ? pos[0] : i == 1 ? pos[1] : pos[2];
        if (p.slots) p.slots[r0 + i] = i == 0 ? slot[0] : i == 1 ? slot[1] : slot[2];
      }
    }
  };
  // four token rows to a thread, or one page entry; rows behind the last token get -1
  const int at = blockIdx.x * kThreads + tid, all = gridDim.x * kThreads, row_items = (p.max_tokens + 3) >> 2;
  for (int64_t item = at; item < int64_t(row_items) + num_entries; item += all) {
    if (item < row_items) {
      write_rows(int(item) * 4);
      continue;
    }
    const int e = int(item - row_items);
    const int b = owner(pages, p.batch, e), j = e - pages[b];
    const int id = checked(read_id(b, j));
    if (j >= fresh_from[b]) p.table[b * p.t_s + j] = id;
    p.kv_indices[e] = id;
  }
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_build_page_table(
    const int32_t* seq_lens, const int32_t* new_lens, int32_t batch, int32_t page_size,
    int32_t* block_table, int64_t table_stride, int32_t max_pages, int32_t num_pages,
    const int32_t* free_pages, int32_t max_free, const int32_t* free_count, int32_t* free_left,
    int32_t* kv_indptr, int32_t* kv_indices, int64_t max_entries, int32_t* kv_last_page_len,
    int32_t* qo_indptr, int32_t* batch_indices, int32_t* positions, int64_t* slots,
    int64_t max_tokens, void* stream) {
  BSKV_NVTX_RANGE("bskv_build_page_table");
  const char* who = "build_page_table";
  if (batch < 0 || page_size < 1 || max_pages < 0 || num_pages < 0 || max_free < 0 || max_tokens < 0) {
    set_error("%s: batch=%d page_size=%d max_pages=%d num_pages=%d max_free=%d max_tokens=%lld", who, batch,
              page_size, max_pages, num_pages, max_free, (long long)max_tokens);
    return BSKV_ERR_INVALID_ARG;
  }
  if (batch > kMaxBatch) { set_error("%s: %d requests (max %d)", who, batch, kMaxBatch); return BSKV_ERR_UNSUPPORTED; }
  const int64_t per_request = int64_t(max_pages) * page_size;
  if (per_request > INT32_MAX - page_size || per_request * std::max(batch, 1) > INT32_MAX || max_tokens > INT32_MAX - 4) {
    set_error("%s: %d requests of %d pages of %d tokens (%lld rows): token numbers exceed 31 bits", who, batch,
              max_pages, page_size, (long long)max_tokens);
    return BSKV_ERR_UNSUPPORTED;
  }
  if (max_entries < int64_t(batch) * max_pages) {
    set_error("%s: kv_indices of %lld entries for %d requests of up to %d pages", who, (long long)max_entries, batch, max_pages);
    return BSKV_ERR_INVALID_ARG;
  }
  if (!kv_indptr || !qo_indptr || (batch > 0 && (!seq_lens || !kv_last_page_len)) ||
      (batch > 0 && max_pages > 0 && (!block_table || !kv_indices)) || (max_tokens > 0 && (!batch_indices || !positions))) {
    set_error("%s: NULL argument", who);
    return BSKV_ERR_INVALID_ARG;
  }
  if (free_pages && (!free_count || !free_left)) { set_error("%s: free_pages need free_count and free_left", who); return BSKV_ERR_INVALID_ARG; }
  if (free_pages && free_count == free_left) { set_error("%s: free_count and free_left must be different memory", who); return BSKV_ERR_INVALID_ARG; }
  if (batch > 0 && max_pages > 0 && table_stride < max_pages && batch > 1) {
    set_error("%s: block_table stride %lld below %d pages", who, (long long)table_stride, max_pages);
    return BSKV_ERR_INVALID_ARG;
  }
  if (!aligned16(batch_indices) || !aligned16(positions) || !aligned16(slots)) {
    set_error("%s: batch_indices, positions and slots must be 16-byte aligned", who);
    return BSKV_ERR_INVALID_ARG;
  }
  const uintptr_t words = reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(new_lens) |
                          reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(free_pages) |
                          reinterpret_cast<uintptr_t>(free_count) | reinterpret_cast<uintptr_t>(free_left) |
                          reinterpret_cast<uintptr_t>(kv_indptr) | reinterpret_cast<uintptr_t>(kv_indices) |
                          reinterpret_cast<uintptr_t>(kv_last_page_len) | reinterpret_cast<uintptr_t>(qo_indptr);
  if (words & 3) { set_error("%s: index arrays must be 4-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  PageTableParams p{};
  p.lens = seq_lens; p.news = new_lens;
  p.table = block_table; p.t_s = table_stride;
  p.batch = batch; p.max_pages = max_pages; p.num_pages = num_pages;
  p.page_size = FastDiv(page_size);
  p.free_pages = free_pages; p.free_count = free_count; p.max_free = max_free;
  p.free_left = free_pages ? free_left : nullptr;
  p.kv_indptr = kv_indptr; p.kv_indices = kv_indices; p.kv_last_page_len = kv_last_page_len; p.qo_indptr = qo_indptr;
  p.batch_indices = batch_indices; p.positions = positions; p.slots = slots; p.max_tokens = int(max_tokens);
  if (bskv_status s = status_args(&p.st)) return s;
  const size_t smem = sizeof(int) * (5 * size_t(batch) + 3);
  static std::atomic<int> allowed[64];
  if (bskv_status s = allow_smem(reinterpret_cast<const void*>(page_table_kernel), smem, allowed, "build_page_table: cudaFuncSetAttribute"))
    return s;
  // A thread for every page entry that there may be and for every four rows, on at most two CTAs per SM.
  const int64_t threads = std::max<int64_t>(int64_t(batch) * max_pages + (max_tokens + 3) / 4, 1);
  const unsigned grid = unsigned(std::min<int64_t>((threads + kThreads - 1) / kThreads, 304));
  page_table_kernel<<<grid, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
  return cuda_check(cudaGetLastError(), "build_page_table launch");
}
