// Queries and keys normalised per head and rotated, keys and values appended to the 16-bit paged cache.
//
// Mathematics, per token and head, in fp32, rounded once:
//   y_d = x_d w_d / sqrt(mean_d(x_d^2) + eps)              (x_d where there is no weight)
//   (a, b) of rotary pair i -> (a cos_i - b sin_i, b cos_i + a sin_i) over the first `rot` dims,
// pairs (i, i + rot / 2) in the half layout and (2i, 2i + 1) interleaved; v is copied.
//
// Bound by memory: every row is read and written once. A warp takes one token (or, where tokens are few, a
// batch of its rows): its heads share the place in the cache and the angles, with which a lane's eight values
// need two factors each,
//   y_d = r (x_d A_d + x_partner B_d),  A_d = w_d cos, B_d = -+ w_partner sin.
// Rows come by asynchronous copies through shared memory, a batch ahead, and a lane takes from there two groups of
// four values whose partners it has too, so that only the mean needs other lanes. What is left to watch is the
// number of instructions: with partners by shuffles and factors made per batch, 165 for two rows of 128 dims, 32000
// tokens of 48 heads took 157 us; so, with 130, they take 127 (6.4 TB/s).
#include <algorithm>
#include <type_traits>

#include "cache_common.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSms = 152;
constexpr int kCtasPerSm = 3;  // 2: 131 us, and 39 instead of 33 for 64 dims; 4 CTAs spill: 208
constexpr int kBatch = 4;  // rows of a lane per batch
constexpr int kStages = 3;
constexpr int kUnroll = 2;

struct NormRopeParams {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_s0, q_s1, k_s0, k_s1, v_s0, v_s1, o_s0, o_s1;
  const void *q_weight, *k_weight;
  const int32_t *batch_indices, *positions, *pos_ids, *kv_indptr, *kv_indices;
  int64_t nnz;
  int hq, hkv, batch, rot, neox, cos_bf16;
  int64_t num_pages, max_seq_len;
  FastDiv page_size;
  void* cache;
  int64_t c_s0, c_s1, c_s2, c_s3;
  const void* cos_sin;
  float eps;
  int q_batches, k_batches, batches;  // of a token
  int span, num_tasks;                // batches of a task; tasks in all
  FastDiv by_token;                   // tasks of a token
  StatusArgs st;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Four consecutive angles of the table, cos from `at` on or sin.
__device__ __forceinline__ float4 angles(const NormRopeParams& p, int64_t at) {
  if (p.cos_bf16) {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.cos_sin) + at));
    return make_float4(__uint_as_float(c.x << 16), __uint_as_float(c.x & 0xffff0000u), __uint_as_float(c.y << 16),
                       __uint_as_float(c.y & 0xffff0000u));
  }
  return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.cos_sin) + at));
}

// A lane's eight values are two groups of four, from `lo` and from `hi` on. In the half layout the
// partner of value e of one is value e of the other, interleaved they are neighbours; values that do not rotate have
// the factors (w, 0).
template <typename T, bool HALF>
__device__ __forceinline__ void factors(const NormRopeParams& p, const void* weight, int64_t at, int lo, int hi,
                                        bool rotated, float (&A)[8], float (&B)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    A[e] = 1.f;
    B[e] = 0.f;
  }
  if (weight) {
    const T* w = static_cast<const T*>(weight);
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(w + lo)), b = __ldg(reinterpret_cast<const uint2*>(w + hi));
    unpack8<T>(make_uint4(a.x, a.y, b.x, b.y), A);
  }
  if (!rotated) return;
  const int half = p.rot >> 1;
  const int64_t base = at * p.rot + (HALF ? lo : lo >> 1);
  const float4 c4 = angles(p, base), s4 = angles(p, base + half);
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = HALF ? e : 2 * e, j = HALF ? e + 4 : 2 * e + 1;
    B[i] = -A[j] * s[e];
    B[j] = A[i] * s[e];
    A[i] *= c[e];
    A[j] *= c[e];
  }
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}

// HALF: half layout.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // rows of a warp's access
  using Mma = MmaOp<T>;
  __shared__ __align__(16) uint8_t ring[kWarps][kStages][kBatch][512];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kLanes, row = lane / kLanes;
  const bool rotated = 8 * sub < p.rot, partly = p.rot < D;
  const int lo = HALF && rotated ? 4 * sub : 8 * sub, hi = HALF && rotated ? (p.rot >> 1) + 4 * sub : 8 * sub + 4;
  const int step = gridDim.x * kWarps;

  // Copies of the batches, kStages - 1 ahead: batch `c` of `c_end` of task `c_task`.
  int c_task = blockIdx.x * kWarps + warp, c_token = 0, c = 0, c_end = 0, c_stage = 0;
  auto begin = [&](int task, int& token, int& from, int& to) {
    int part;
    token = p.by_token.divmod(task, part);
    from = part * p.span;
    to = min(p.batches, from + p.span);
  };
  if (c_task < p.num_tasks) begin(c_task, c_token, c, c_end);
  auto issue = [&]() {
    if (c_task < p.num_tasks) {
      const int kind = c < p.q_batches ? 0 : c < p.q_batches + p.k_batches ? 1 : 2;
      const T* from = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v);
      const int64_t s0 = kind == 0 ? p.q_s0 : kind == 1 ? p.k_s0 : p.v_s0, s1 = kind == 0 ? p.q_s1 : kind == 1 ? p.k_s1 : p.v_s1;
      const int before = kind == 0 ? 0 : kind == 1 ? p.q_batches : p.q_batches + p.k_batches;
      const int heads = kind ? p.hkv : p.hq, g = (c - before) * kBatch * kRows + row;
      from += c_token * s0 + g * s1 + 8 * sub;
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (g + r * kRows < heads) cp_async_16(&ring[warp][c_stage][r][16 * lane], from);
        from += kRows * s1;
      }
      if (++c == c_end) {
        c_task += step;
        if (c_task < p.num_tasks) begin(c_task, c_token, c, c_end);
      }
    }
    cp_async_commit();
    c_stage = c_stage + 1 == kStages ? 0 : c_stage + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  int task = blockIdx.x * kWarps + warp, b = -1, pos = 0, at = 0, stage = 0;
  auto indices = [&](int i, int& b_, int& pos_, int& at_) {
    b_ = -1;
    if (i >= p.num_tasks) return;
    const int t = p.by_token.div(i);
    b_ = __ldg(p.batch_indices + t);
    pos_ = __ldg(p.positions + t);
    at_ = p.pos_ids ? __ldg(p.pos_ids + t) : pos_;
  };
  indices(task, b, pos, at);
  while (task < p.num_tasks) {
    int token, i0, i1;
    begin(task, token, i0, i1);
    // the next task's indices are on their way while this one is computed
    const int next = task + step;
    int next_b = -1, next_pos = 0, next_at = 0;
    indices(next, next_b, next_pos, next_at);
    const bool in_table = !p.rot || (at >= 0 && at < p.max_seq_len);
    if (b >= 0 && !in_table && lane == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    const bool live = b >= 0 && in_table;
    T* cache = nullptr;  // the token's first K row
    if (live && i1 > p.q_batches) {
      if (b < p.batch && pos >= 0) {
        int slot;
        const int j = p.page_size.divmod(pos, slot);
        const int first = __ldg(p.kv_indptr + b), end = __ldg(p.kv_indptr + b + 1);
        const int page = j < end - first ? __ldg(p.kv_indices + first + j) : -1;
        if (page >= 0 && page < p.num_pages) cache = static_cast<T*>(p.cache) + page * p.c_s0 + slot * p.c_s3;
      }
      if (!cache && lane == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    }
    float A[8], B[8];
    for (int i = i0; i < i1; ++i) {
      const int kind = i < p.q_batches ? 0 : i < p.q_batches + p.k_batches ? 1 : 2;
      const void* weight = kind ? p.k_weight : p.q_weight;
      if (live && kind < 2 && (i == i0 || i == p.q_batches)) factors<T, HALF>(p, weight, at, lo, hi, rotated, A, B);
      issue();
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const int before = kind == 0 ? 0 : kind == 1 ? p.q_batches : p.q_batches + p.k_batches;
      const int heads = kind ? p.hkv : p.hq, g0 = (i - before) * kBatch * kRows;
      T* out = kind ? cache : static_cast<T*>(p.q_out) + token * p.o_s0;
      if (live && out) {
        const int64_t s1 = kind ? p.c_s2 : p.o_s1;
        out += (g0 + row) * s1 + (kind == 2 ? p.c_s1 : 0);
        const uint8_t* in = &ring[warp][stage][0][row * 2 * D];
#pragma unroll kUnroll
        for (int r = 0; r < kBatch; ++r) {
          if (g0 + r * kRows >= heads) break;
          uint2 a, z;
          if constexpr (HALF) {
            a = *reinterpret_cast<const uint2*>(in + 512 * r + 2 * lo);
            z = *reinterpret_cast<const uint2*>(in + 512 * r + 2 * hi);
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(in + 512 * r + 2 * lo);
            a = make_uint2(x.x, x.y);
            z = make_uint2(x.z, x.w);
          }
          if (kind < 2) {
            float x[8];
            unpack8<T>(make_uint4(a.x, a.y, z.x, z.y), x);
            float f = 1.f;
            if (weight) {
              float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 8; e += 2) s2 = ffma2(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), s2);
              float ss = s2.x + s2.y;
#pragma unroll
              for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
              f = rsqrtf(ss * (1.f / D) + p.eps);
            }
            float y[8];  // partners
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = HALF ? x[e ^ 4] : x[e ^ 1];
            if (partly && !rotated) {  // times B = 0, whatever x is
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 v = fmul2(make_float2(f, f), ffma2(make_float2(x[e], x[e + 1]), make_float2(A[e], A[e + 1]),
                                                              fmul2(make_float2(y[e], y[e + 1]), make_float2(B[e], B[e + 1]))));
              (e < 4 ? e == 0 ? a.x : a.y : e == 4 ? z.x : z.y) = Mma::pack(v.x, v.y);
            }
          }
          if (g0 + row + r * kRows < heads) {
            if constexpr (HALF) {
              *reinterpret_cast<uint2*>(out + lo) = a;
              *reinterpret_cast<uint2*>(out + hi) = z;
            } else {
              *reinterpret_cast<uint4*>(out + lo) = make_uint4(a.x, a.y, z.x, z.y);
            }
          }
          out += kRows * s1;
        }
      }
      __syncwarp();  // the stage is read before it is filled again
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    task = next;
    b = next_b;
    pos = next_pos;
    at = next_at;
  }
}

template <typename T>
bskv_status launch(NormRopeParams& p, int D, cudaStream_t st) {
  const int rows = kBatch * (32 / (D / 8));
  p.q_batches = (p.hq + rows - 1) / rows;
  p.k_batches = (p.hkv + rows - 1) / rows;
  p.batches = p.q_batches + 2 * p.k_batches;
  // a warp takes a token, or single batches while there are fewer tokens than two thirds of the warps (batches
  // against tokens, 32 + 2 * 8 heads of 128 dims: 512 tokens 4.8 and 10.1 us, 1824 14.0 and 14.4, 2736 18.6 and 17.5,
  // 7296 40.8 and 32.5)
  const int64_t warps = int64_t(kSms) * kCtasPerSm * kWarps;
  p.span = p.nnz * 3 >= warps * 2 ? p.batches : 1;
  const int per_token = (p.batches + p.span - 1) / p.span;
  if (p.nnz > INT32_MAX / 2 / per_token) {
    set_error("norm_rope_append_paged: %lld rows of %d + 2 * %d heads are too many", (long long)p.nnz, p.hq, p.hkv);
    return BSKV_ERR_UNSUPPORTED;
  }
  p.num_tasks = int(p.nnz) * per_token;
  p.by_token = FastDiv(per_token);
  const unsigned grid = unsigned(std::min<int64_t>((p.num_tasks + kWarps - 1) / kWarps, warps / kWarps));
  auto kern = D == 128 ? (p.neox ? norm_rope_kernel<T, 128, true> : norm_rope_kernel<T, 128, false>)
                       : (p.neox ? norm_rope_kernel<T, 64, true> : norm_rope_kernel<T, 64, false>);
  kern<<<grid, kThreads, 0, st>>>(p);
  return cuda_check(cudaGetLastError(), "norm_rope_append_paged launch");
}

}  // namespace
}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_norm_rope_append_paged(
    const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
    const int64_t* v_strides, int32_t dtype, int64_t nnz, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, const void* q_weight, const void* k_weight, float eps, const void* cos_sin,
    int32_t cos_sin_dtype, int64_t max_seq_len, int32_t rotary_dim, int32_t is_neox,
    const int32_t* pos_ids, const int32_t* batch_indices, const int32_t* positions,
    const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch, int32_t page_size,
    int64_t num_pages, void* q_out, const int64_t* q_out_strides, void* kv_cache,
    const int64_t* kv_strides, void* stream) {
  BSKV_NVTX_RANGE("bskv_norm_rope_append_paged");
  const char* who = "norm_rope_append_paged";
  const bool has_q = q || q_out, has_kv = k || v || kv_cache;
  if (dtype != BSKV_BF16 && dtype != BSKV_FP16) { set_error("%s: dtype %s unsupported", who, dtype_name(dtype)); return BSKV_ERR_UNSUPPORTED; }
  if (head_dim != 64 && head_dim != 128) { set_error("%s: head_dim %d not in {64,128}", who, head_dim); return BSKV_ERR_UNSUPPORTED; }
  if (nnz < 0 || batch < 0 || page_size < 1 || num_pages < 0 || (has_q && num_qo_heads < 1) || (has_kv && num_kv_heads < 1)) {
    set_error("%s: nnz=%lld num_qo_heads=%d num_kv_heads=%d batch=%d page_size=%d num_pages=%lld", who, (long long)nnz,
              num_qo_heads, num_kv_heads, batch, page_size, (long long)num_pages);
    return BSKV_ERR_INVALID_ARG;
  }
  if (!has_q && !has_kv) { set_error("%s: neither queries nor keys and values", who); return BSKV_ERR_INVALID_ARG; }
  if (nnz > INT32_MAX || num_pages > INT32_MAX || num_qo_heads > 65535 || num_kv_heads > 65535) {
    set_error("%s: nnz=%lld num_pages=%lld num_qo_heads=%d num_kv_heads=%d", who, (long long)nnz, (long long)num_pages, num_qo_heads, num_kv_heads);
    return BSKV_ERR_UNSUPPORTED;
  }
  if (rotary_dim < 0 || rotary_dim > head_dim) { set_error("%s: rotary_dim %d outside [0, %d]", who, rotary_dim, head_dim); return BSKV_ERR_INVALID_ARG; }
  if (rotary_dim % 16) { set_error("%s: rotary_dim %d must be a multiple of 16", who, rotary_dim); return BSKV_ERR_UNSUPPORTED; }
  if (cos_sin_dtype != BSKV_FP32 && cos_sin_dtype != BSKV_BF16) { set_error("%s: cos_sin dtype %s unsupported", who, dtype_name(cos_sin_dtype)); return BSKV_ERR_UNSUPPORTED; }
  if (!(eps >= 0.f)) { set_error("%s: eps=%g", who, double(eps)); return BSKV_ERR_INVALID_ARG; }
  if (nnz == 0) return BSKV_OK;
  if (rotary_dim && (!cos_sin || max_seq_len < 1 || !aligned16(cos_sin))) { set_error("%s: cos_sin must be a 16-byte aligned table", who); return BSKV_ERR_INVALID_ARG; }
  if (!batch_indices || !positions) { set_error("%s: NULL argument", who); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(q_weight) || !aligned16(k_weight)) { set_error("%s: weights must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  NormRopeParams p{};
  auto strides_ok = [&](const char* name, const void* x, const int64_t* s, int n) {
    if (!x || !s || !aligned16(x)) { set_error("%s: %s must be a 16-byte aligned tensor", who, name); return false; }
    for (int i = 0; i < n; ++i)
      if (s[i] < 0 || s[i] % 8) { set_error("%s: stride %d of %s (%lld elements) must be a multiple of 16 bytes", who, i, name, (long long)s[i]); return false; }
    return true;
  };
  if (has_q) {
    if (!strides_ok("q", q, q_strides, 2) || !strides_ok("q_out", q_out, q_out_strides, 2)) return BSKV_ERR_INVALID_ARG;
    p.q = q; p.q_s0 = q_strides[0]; p.q_s1 = q_strides[1];
    p.q_out = q_out; p.o_s0 = q_out_strides[0]; p.o_s1 = q_out_strides[1];
    p.hq = num_qo_heads; p.q_weight = q_weight;
  }
  if (has_kv) {
    if (!strides_ok("k", k, k_strides, 2) || !strides_ok("v", v, v_strides, 2) || !strides_ok("kv_cache", kv_cache, kv_strides, 4)) return BSKV_ERR_INVALID_ARG;
    if (!kv_indptr || !kv_indices) { set_error("%s: NULL page table", who); return BSKV_ERR_INVALID_ARG; }
    p.k = k; p.k_s0 = k_strides[0]; p.k_s1 = k_strides[1];
    p.v = v; p.v_s0 = v_strides[0]; p.v_s1 = v_strides[1];
    p.hkv = num_kv_heads; p.k_weight = k_weight;
    p.cache = kv_cache; p.c_s0 = kv_strides[0]; p.c_s1 = kv_strides[1]; p.c_s2 = kv_strides[2]; p.c_s3 = kv_strides[3];
  }
  if ((reinterpret_cast<uintptr_t>(batch_indices) | reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(pos_ids) |
       reinterpret_cast<uintptr_t>(kv_indptr) | reinterpret_cast<uintptr_t>(kv_indices)) & 3) {
    set_error("%s: index arrays must be 4-byte aligned", who);
    return BSKV_ERR_INVALID_ARG;
  }
  p.batch_indices = batch_indices; p.positions = positions; p.pos_ids = pos_ids;
  p.kv_indptr = kv_indptr; p.kv_indices = kv_indices;
  p.nnz = nnz; p.batch = batch; p.num_pages = num_pages; p.page_size = FastDiv(page_size);
  p.rot = rotary_dim; p.neox = is_neox != 0; p.cos_sin = cos_sin; p.cos_bf16 = cos_sin_dtype == BSKV_BF16;
  p.max_seq_len = max_seq_len; p.eps = eps;
  if (bskv_status s = status_args(&p.st)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == BSKV_BF16 ? launch<__nv_bfloat16>(p, head_dim, st) : launch<__half>(p, head_dim, st);
}
