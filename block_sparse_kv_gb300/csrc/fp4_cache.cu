// Writing K and V rows into a 4-bit paged cache, and reading them back.
//
// Mathematics: a row's head_dim values are cut into blocks of 32; a block of largest magnitude
// m gets the scale X = 2^(floor(log2 m) - 2) and each value v becomes the E2M1 number nearest
// to v / X (ties to even, at most 6): the OCP Microscaling conversion. X is a power of two, so
// v / X is exact in fp32 and one rounding, cvt.rn.satfinite.e2m1x2, is made per value.
//
// Both directions are HBM streams (2 bytes and 17/32 bytes a value). A lane owns 8 values: one
// 16-byte load or store on the 16-bit side, 4 bytes of codes on the other; the four lanes of a
// block find its maximum with two shuffles. A lane issues the loads of kUnroll chunks, and the
// index chains of their rows (request, position -> page table -> page), before it converts any.
#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kUnroll = 4;     // 8-value chunks per lane
constexpr int kThreads = 256;

struct Fp4CacheParams {
  void* rows[2];  // K, V: 16-bit (or fp32) rows, [nnz, heads, D]
  int64_t r_s0[2], r_s1[2];
  uint8_t* codes;
  int64_t c_s0, c_s1, c_s2, c_s3;  // bytes
  uint8_t* scales;
  int64_t s_s0, s_s1, s_s2;  // bytes
  const int32_t* batch_indices;
  const int32_t* positions;
  const int32_t* indptr;
  const int32_t* indices;
  int32_t batch, page_size;
  int64_t num_pages;
  int64_t chunks;     // nnz * 2 * heads * D / 8
  int32_t per_token;  // 2 * heads * D / 8
  int32_t heads;
  StatusArgs st;
};

// Where a chunk's row lies: token, K or V, head, first value.
struct ChunkAt {
  int64_t token;
  int32_t which, head, d;
};

template <int D>
__device__ __forceinline__ ChunkAt chunk_place(const Fp4CacheParams& p, int64_t id) {
  ChunkAt a;
  a.token = id / p.per_token;
  const int32_t r = int32_t(id - a.token * p.per_token);
  const int32_t row = r / (D / 8);
  a.d = (r % (D / 8)) * 8;
  a.which = row >= p.heads ? 1 : 0;
  a.head = row - a.which * p.heads;
  return a;
}

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_float2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 to_float2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fp4_append_kernel(const Fp4CacheParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t base = (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 * kUnroll);
  uint4 x[kUnroll];
  ChunkAt at[kUnroll];
  int32_t page[kUnroll], slot[kUnroll];
  bool live[kUnroll], ok[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t id = base + j * 32 + lane;
    live[j] = id < p.chunks;
    x[j] = make_uint4(0, 0, 0, 0);
    if (!live[j]) continue;
    at[j] = chunk_place<D>(p, id);
    const T* row = static_cast<const T*>(p.rows[at[j].which]) + at[j].token * p.r_s0[at[j].which] +
                   at[j].head * p.r_s1[at[j].which] + at[j].d;
    x[j] = __ldcs(reinterpret_cast<const uint4*>(row));
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    ok[j] = live[j] && page_slot(p.indptr, p.indices, p.batch, p.page_size, p.num_pages,
                                 __ldg(p.batch_indices + at[j].token),
                                 __ldg(p.positions + at[j].token), page[j], slot[j]);
    if (live[j] && !ok[j]) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    float2 v[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = to_float2<T>(w[i]);
      top = max(top, max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t code = e8m0_of_max(top);
    const float inv = e8m0_inverse(code == 255u ? 127u : code);
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) packed |= cvt_e2m1x2(v[i].x * inv, v[i].y * inv) << (8 * i);
    if (!ok[j]) continue;
    uint8_t* c = p.codes + page[j] * p.c_s0 + at[j].which * p.c_s1 + at[j].head * p.c_s2 +
                 slot[j] * p.c_s3 + at[j].d / 2;
    *reinterpret_cast<uint32_t*>(c) = packed;
    if ((lane & 3) == 0)
      p.scales[page[j] * p.s_s0 + at[j].which * p.s_s1 + at[j].head * p.s_s2 +
               slot[j] * (D / kFp4Block) + at[j].d / kFp4Block] = uint8_t(code);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* dst, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(dst), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&v)[8]) {
  using M = MmaOp<__nv_bfloat16>;
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(M::pack(v[0], v[1]), M::pack(v[2], v[3]),
                                                   M::pack(v[4], v[5]), M::pack(v[6], v[7])));
}
template <>
__device__ __forceinline__ void store8<__half>(__half* dst, const float (&v)[8]) {
  using M = MmaOp<__half>;
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(M::pack(v[0], v[1]), M::pack(v[2], v[3]),
                                                   M::pack(v[4], v[5]), M::pack(v[6], v[7])));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fp4_read_kernel(const Fp4CacheParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t base = (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 * kUnroll);
  ChunkAt at[kUnroll];
  uint32_t w[kUnroll], code[kUnroll];
  bool ok[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t id = base + j * 32 + lane;
    const bool live = id < p.chunks;
    int32_t page = 0, slot = 0;
    if (live) at[j] = chunk_place<D>(p, id);
    ok[j] = live && page_slot(p.indptr, p.indices, p.batch, p.page_size, p.num_pages,
                              __ldg(p.batch_indices + at[j].token),
                              __ldg(p.positions + at[j].token), page, slot);
    if (live && !ok[j]) record_error(p.st, BSKV_ERR_DEVICE_INDEX);
    if (!ok[j]) continue;
    w[j] = *reinterpret_cast<const uint32_t*>(p.codes + page * p.c_s0 + at[j].which * p.c_s1 +
                                              at[j].head * p.c_s2 + slot * p.c_s3 + at[j].d / 2);
    code[j] = p.scales[page * p.s_s0 + at[j].which * p.s_s1 + at[j].head * p.s_s2 +
                       slot * (D / kFp4Block) + at[j].d / kFp4Block];
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    if (!ok[j]) continue;
    uint32_t h[4];
    cvt_e2m1x8(w[j], h);
    const float f = e8m0_value(code[j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
      v[2 * i] = a.x * f;
      v[2 * i + 1] = a.y * f;
    }
    store8<T>(static_cast<T*>(p.rows[at[j].which]) + at[j].token * p.r_s0[at[j].which] +
                  at[j].head * p.r_s1[at[j].which] + at[j].d, v);
  }
}

// Argument checks and parameters shared by the two entry points.
bskv_status prepare(const char* who, const void* k, const int64_t* k_strides, const void* v,
                    const int64_t* v_strides, int32_t esz, int64_t nnz, int32_t num_kv_heads,
                    int32_t head_dim, const int32_t* batch_indices, const int32_t* positions,
                    const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch,
                    int32_t page_size, int64_t num_pages, const void* kv_codes,
                    const int64_t* codes_strides, const void* kv_scales,
                    const int64_t* scales_strides, Fp4CacheParams* p) {
  if (nnz < 0 || num_kv_heads < 1 || batch < 0 || num_pages < 0) {
    set_error("%s: nnz=%lld num_kv_heads=%d batch=%d num_pages=%lld", who, (long long)nnz,
              num_kv_heads, batch, (long long)num_pages);
    return BSKV_ERR_INVALID_ARG;
  }
  if (head_dim != 64 && head_dim != 128) { set_error("%s: head_dim %d not in {64,128}", who, head_dim); return BSKV_ERR_UNSUPPORTED; }
  if (page_size < 1) { set_error("%s: page_size %d", who, page_size); return BSKV_ERR_INVALID_ARG; }
  if (!fp4_page_size(page_size)) { set_error("%s: page_size %d unsupported (8 or a multiple of 16)", who, page_size); return BSKV_ERR_UNSUPPORTED; }
  if (num_pages > INT32_MAX || int64_t(num_kv_heads) * head_dim / 4 > INT32_MAX) {
    set_error("%s: too large", who);
    return BSKV_ERR_UNSUPPORTED;
  }
  if (nnz == 0) return BSKV_OK;
  if (!k || !v || !k_strides || !v_strides || !batch_indices || !positions || !kv_indptr ||
      !kv_indices || !codes_strides || !scales_strides) {
    set_error("%s: NULL argument", who);
    return BSKV_ERR_INVALID_ARG;
  }
  if (bskv_status s = check_fp4_cache(who, kv_codes, codes_strides, kv_scales, scales_strides)) return s;
  if (!aligned16(k) || !aligned16(v)) { set_error("%s: rows must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i) {
    if ((k_strides[i] * esz) % 16 || (v_strides[i] * esz) % 16 || k_strides[i] < 0 || v_strides[i] < 0) {
      set_error("%s: row strides must be multiples of 16 bytes", who);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  *p = Fp4CacheParams{};
  p->rows[0] = const_cast<void*>(k); p->rows[1] = const_cast<void*>(v);
  p->r_s0[0] = k_strides[0]; p->r_s1[0] = k_strides[1];
  p->r_s0[1] = v_strides[0]; p->r_s1[1] = v_strides[1];
  p->codes = static_cast<uint8_t*>(const_cast<void*>(kv_codes));
  p->c_s0 = codes_strides[0]; p->c_s1 = codes_strides[1]; p->c_s2 = codes_strides[2]; p->c_s3 = codes_strides[3];
  p->scales = static_cast<uint8_t*>(const_cast<void*>(kv_scales));
  p->s_s0 = scales_strides[0]; p->s_s1 = scales_strides[1]; p->s_s2 = scales_strides[2];
  p->batch_indices = batch_indices; p->positions = positions;
  p->indptr = kv_indptr; p->indices = kv_indices;
  p->batch = batch; p->page_size = page_size; p->num_pages = num_pages;
  p->heads = num_kv_heads;
  p->per_token = 2 * num_kv_heads * (head_dim / 8);
  p->chunks = nnz * p->per_token;
  if ((p->chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll) > INT32_MAX) {
    set_error("%s: too many rows", who);
    return BSKV_ERR_UNSUPPORTED;
  }
  return status_args(&p->st);
}

unsigned grid_of(const Fp4CacheParams& p) {
  return unsigned((p.chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll));
}

}  // namespace

bskv_status check_fp4_cache(const char* who, const void* kv_codes, const int64_t* codes_strides,
                            const void* kv_scales, const int64_t* scales_strides) {
  if (!kv_codes || !kv_scales || !codes_strides || !scales_strides) { set_error("%s: NULL cache", who); return BSKV_ERR_INVALID_ARG; }
  if (!aligned16(kv_codes) || !aligned16(kv_scales)) { set_error("%s: the cache must be 16-byte aligned", who); return BSKV_ERR_INVALID_ARG; }
  for (int i = 0; i < 4; ++i) {
    if (codes_strides[i] <= 0 || codes_strides[i] % 16) {
      set_error("%s: codes stride %d (%lld) must be a positive multiple of 16 bytes", who, i, (long long)codes_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  for (int i = 0; i < 3; ++i) {
    if (scales_strides[i] <= 0 || scales_strides[i] % 16) {
      set_error("%s: scales stride %d (%lld) must be a positive multiple of 16 bytes", who, i, (long long)scales_strides[i]);
      return BSKV_ERR_INVALID_ARG;
    }
  }
  return BSKV_OK;
}

}  // namespace bskv

using namespace bskv;

extern "C" bskv_status bskv_quantize_fp4_append_paged(
    const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides, int32_t dtype,
    int64_t nnz, int32_t num_kv_heads, int32_t head_dim, const int32_t* batch_indices,
    const int32_t* positions, const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch,
    int32_t page_size, int64_t num_pages, void* kv_codes, const int64_t* codes_strides,
    void* kv_scales, const int64_t* scales_strides, void* stream) {
  BSKV_NVTX_RANGE("bskv_quantize_fp4_append_paged");
  if (dtype != BSKV_BF16 && dtype != BSKV_FP16) { set_error("quantize_fp4_append_paged: dtype %s unsupported", dtype_name(dtype)); return BSKV_ERR_UNSUPPORTED; }
  Fp4CacheParams p;
  if (bskv_status s = prepare("quantize_fp4_append_paged", k, k_strides, v, v_strides, 2, nnz,
                              num_kv_heads, head_dim, batch_indices, positions, kv_indptr,
                              kv_indices, batch, page_size, num_pages, kv_codes, codes_strides,
                              kv_scales, scales_strides, &p))
    return s;
  if (nnz == 0) return BSKV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == BSKV_BF16;
  if (head_dim == 128) {
    if (bf) fp4_append_kernel<__nv_bfloat16, 128><<<grid_of(p), kThreads, 0, st>>>(p);
    else fp4_append_kernel<__half, 128><<<grid_of(p), kThreads, 0, st>>>(p);
  } else {
    if (bf) fp4_append_kernel<__nv_bfloat16, 64><<<grid_of(p), kThreads, 0, st>>>(p);
    else fp4_append_kernel<__half, 64><<<grid_of(p), kThreads, 0, st>>>(p);
  }
  return cuda_check(cudaGetLastError(), "quantize_fp4_append_paged launch");
}

extern "C" bskv_status bskv_dequantize_fp4_paged(
    const void* kv_codes, const int64_t* codes_strides, const void* kv_scales,
    const int64_t* scales_strides, const int32_t* batch_indices, const int32_t* positions,
    const int32_t* kv_indptr, const int32_t* kv_indices, int32_t batch, int32_t page_size,
    int64_t num_pages, void* k_out, const int64_t* k_strides, void* v_out,
    const int64_t* v_strides, int32_t dtype, int64_t nnz, int32_t num_kv_heads, int32_t head_dim,
    void* stream) {
  BSKV_NVTX_RANGE("bskv_dequantize_fp4_paged");
  if (dtype != BSKV_BF16 && dtype != BSKV_FP16 && dtype != BSKV_FP32) { set_error("dequantize_fp4_paged: dtype %s unsupported", dtype_name(dtype)); return BSKV_ERR_UNSUPPORTED; }
  Fp4CacheParams p;
  if (bskv_status s = prepare("dequantize_fp4_paged", k_out, k_strides, v_out, v_strides,
                              dtype == BSKV_FP32 ? 4 : 2, nnz, num_kv_heads, head_dim,
                              batch_indices, positions, kv_indptr, kv_indices, batch, page_size,
                              num_pages, kv_codes, codes_strides, kv_scales, scales_strides, &p))
    return s;
  if (nnz == 0) return BSKV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = grid_of(p);
  if (head_dim == 128) {
    if (dtype == BSKV_BF16) fp4_read_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(p);
    else if (dtype == BSKV_FP16) fp4_read_kernel<__half, 128><<<grid, kThreads, 0, st>>>(p);
    else fp4_read_kernel<float, 128><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (dtype == BSKV_BF16) fp4_read_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(p);
    else if (dtype == BSKV_FP16) fp4_read_kernel<__half, 64><<<grid, kThreads, 0, st>>>(p);
    else fp4_read_kernel<float, 64><<<grid, kThreads, 0, st>>>(p);
  }
  return cuda_check(cudaGetLastError(), "dequantize_fp4_paged launch");
}
