// Queries and keys normalised per head and rotated, keys and values appended to the 16-bit paged cache.
//
// Mathematics, per token and head, in fp32, rounded once:
//   y_d = x_d w_d / sqrt(mean_d(x_d^2) + eps)              (x_d where there is no weight)
//   (a, b) of rotary pair i -> (a cos_i - b sin_i, b cos_i + a sin_i) over the first `rot` dims,
// pairs (i, i + rot / 2) in the half layout and (2i, 2i + 1) interleaved; v is copied.
//
// Bound by memory: every row is read and written once. A row is D / 8 lanes of 16 bytes, so that a
// warp's access is whole lines; the mean is a reduction over those lanes and the partner of a half-layout
// pair comes from the lane that holds it. A CTA takes one token at a time: its heads share the angles,
// which a lane keeps in registers, and the place in the cache. A lane reads up to four heads before it
// computes the first.
#include <algorithm>
#include <type_traits>

#include "cache_common.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads that a lane has in flight

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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  using Mma = MmaOp<T>;
  const int sub = threadIdx.x % kLanes, row = threadIdx.x / kLanes, d0 = 8 * sub;
  const int heads = p.hq + 2 * p.hkv;
  const int half = p.rot >> 1;
  const bool rotated = d0 < p.rot, second = p.neox && d0 >= half;
  // lane of the row's that holds the other values of the pairs
  const int partner = (threadIdx.x & 31) - sub + (second ? sub - half / 8 : rotated ? sub + half / 8 : sub);
  for (int64_t t = blockIdx.x; t < p.nnz; t += gridDim.x) {
    const int b = __ldg(p.batch_indices + t);
    if (b < 0) continue;  // a row without a token
    const int pos = __ldg(p.positions + t);
    const int64_t at = p.pos_ids ? __ldg(p.pos_ids + t) : pos;
    int64_t place = -1;  // of the token's K rows in the cache
    if (p.k) {
      if (b < p.batch && pos >= 0) {
        int slot;
        const int j = p.page_size.divmod(pos, slot);
        const int first = __ldg(p.kv_indptr + b), end = __ldg(p.kv_indptr + b + 1);
        const int page = j < end - first ? __ldg(p.kv_indices + first + j) : -1;
        if (page >= 0 && page < p.num_pages) place = page * p.c_s0 + slot * p.c_s3;
      }
      if (place < 0 && threadIdx.x == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    }
    float cs[8], sn[8];
    if (p.rot) {
      if (at < 0 || at >= p.max_seq_len) {
        if (threadIdx.x == 0) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
        continue;
      }
      const int pair = p.neox ? (second ? d0 - half : d0) : d0 >> 1, n = p.neox ? 8 : 4;
      const int64_t base = at * p.rot + pair;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        if (!rotated || i >= n) continue;
        if (p.cos_bf16) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.cos_sin) + base + i));
          const uint2 s = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.cos_sin) + base + half + i));
          cs[i] = __uint_as_float(c.x << 16);
          cs[i + 1] = __uint_as_float(c.x & 0xffff0000u);
          cs[i + 2] = __uint_as_float(c.y << 16);
          cs[i + 3] = __uint_as_float(c.y & 0xffff0000u);
          sn[i] = __uint_as_float(s.x << 16);
          sn[i + 1] = __uint_as_float(s.x & 0xffff0000u);
          sn[i + 2] = __uint_as_float(s.y << 16);
          sn[i + 3] = __uint_as_float(s.y & 0xffff0000u);
        } else {
          const float4 c = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.cos_sin) + base + i));
          const float4 s = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.cos_sin) + base + half + i));
          cs[i] = c.x;
          cs[i + 1] = c.y;
          cs[i + 2] = c.z;
          cs[i + 3] = c.w;
          sn[i] = s.x;
          sn[i + 1] = s.y;
          sn[i + 2] = s.z;
          sn[i + 3] = s.w;
        }
      }
    }
    for (int h0 = row; h0 - row < heads; h0 += kBatch * kRows) {
      uint4 in[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * kRows;
        const T* from = nullptr;
        if (h < p.hq) from = static_cast<const T*>(p.q) + t * p.q_s0 + h * p.q_s1;
        else if (h < p.hq + p.hkv) from = static_cast<const T*>(p.k) + t * p.k_s0 + (h - p.hq) * p.k_s1;
        else if (h < heads) from = static_cast<const T*>(p.v) + t * p.v_s0 + (h - p.hq - p.hkv) * p.v_s1;
        in[i] = from ? *reinterpret_cast<const uint4*>(from + d0) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 - row + i * kRows >= heads) break;  // the same for all rows of the CTA
        const int h = h0 + i * kRows;
        const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
        const void* weight = is_q ? p.q_weight : p.k_weight;
        uint4 out = in[i];
        float x[8];
        unpack8<T>(in[i], x);
        if (p.q_weight || p.k_weight) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (weight) {
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            float w[8];
            unpack8<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + d0)), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
          }
        }
        if (p.rot) {
          if (p.neox) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
            if (rotated) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], cs[e], second ? y[e] * sn[e] : -y[e] * sn[e]);
            }
          } else if (rotated) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = x[2 * e], c = x[2 * e + 1];
              x[2 * e] = fmaf(a, cs[e], -c * sn[e]);
              x[2 * e + 1] = fmaf(c, cs[e], a * sn[e]);
            }
          }
        }
        if (!is_v) out = make_uint4(Mma::pack(x[0], x[1]), Mma::pack(x[2], x[3]), Mma::pack(x[4], x[5]), Mma::pack(x[6], x[7]));
        if (h >= heads) continue;
        if (is_q) {
          *reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + t * p.o_s0 + h * p.o_s1 + d0) = out;
        } else if (place >= 0) {
          const int64_t head = is_v ? (h - p.hq - p.hkv) * p.c_s2 + p.c_s1 : (h - p.hq) * p.c_s2;
          *reinterpret_cast<uint4*>(static_cast<T*>(p.cache) + place + head + d0) = out;
        }
      }
    }
  }
}

template <typename T>
bskv_status launch(const NormRopeParams& p, int D, cudaStream_t st) {
  const unsigned grid = unsigned(std::min<int64_t>(p.nnz, 1 << 20));
  if (D == 128) norm_rope_kernel<T, 128><<<grid, kThreads, 0, st>>>(p);
  else norm_rope_kernel<T, 64><<<grid, kThreads, 0, st>>>(p);
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
  if (num_pages > INT32_MAX || num_qo_heads > 65535 || num_kv_heads > 65535) {
    set_error("%s: num_pages=%lld num_qo_heads=%d num_kv_heads=%d", who, (long long)num_pages, num_qo_heads, num_kv_heads);
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
