// Writing K and V rows into a 4-bit paged cache, and reading them back.
//
// Mathematics: a row's head_dim values are cut into blocks of 32; a block of largest magnitude
// m gets the scale X = 2^(floor(log2 m) - 2) and each value v becomes the E2M1 number nearest
// to v / X (ties to even, at most 6): the OCP Microscaling conversion. X is a power of two, so
// v / X is exact in fp32 and one rounding, cvt.rn.satfinite.e2m1x2, is made per value.
//
// Both directions are HBM streams (2 bytes and 17/32 bytes a value), and what it takes to find a
// row's addresses costs more instructions than the conversion if every thread does it. A thread owns
// half a block of 32 (a chunk): the values 8 e .. 8 e + 7 and 16 + 8 e .. of it for lane parity e, so
// that a pair of lanes reads or writes whole 32-byte sectors; one shuffle finds the block's maximum.
// A CTA of a few thousand chunks makes two tables in shared memory, one entry per thread: the places
// of its tokens (three dependent loads: request and position, page table, page) and of the 2 x heads
// rows of a token. The rows of several prompts, 46 MB of them, take 15.4 us to write and 13.7 us to
// read back.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.h"

namespace bskv {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                   // chunks of 16 values per thread and pass
constexpr int kPass = kThreads * kUnroll;
constexpr int kMaxTokens = kPass / 8 + 2;    // of a CTA: a pass touches at most these (8 chunks a token)
constexpr int kCtas = 4 * 152;               // four per SM: enough CTAs to share long inputs
constexpr int kMaxHeads = 128;

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
  int64_t chunks;     // nnz * 2 * heads * D / 16
  int32_t span;       // chunks of a CTA, a multiple of kPass
  int32_t per_token;  // 2 * heads * D / 16
  uint32_t magic;     // ceil(2^32 / (2 heads)): r / (2 heads) = hi(r * magic) while r * 2 heads < 2^32
  int32_t heads, esz;  // bytes per value of the rows
  StatusArgs st;
};

// Byte offsets of a token in the cache (codes = -1 when it has no place there), and of row r of a
// token (K of every head, then V); `rows` is the row of the CTA's first token on the 16-bit side.
struct TokenAt {
  int64_t codes, scales;
};
struct RowAt {
  const uint8_t* rows;
  int64_t codes, scales;
};
struct Tables {
  TokenAt token[kMaxTokens];
  RowAt row[2 * kMaxHeads];
};

// The CTA's chunks. Chunk j of a thread (j * kThreads + its index) has the same values of its row for
// every j: d .. d + 7 and d + 16 .. d + 23.
template <int D>
struct Chunks {
  int64_t t0;  // first token
  int32_t row0, d, left;
  __device__ __forceinline__ explicit Chunks(const Fp4CacheParams& p) {
    const int64_t base = int64_t(blockIdx.x) * p.span;
    t0 = base / p.per_token;
    const int32_t r = int32_t(base - t0 * p.per_token) + threadIdx.x, c = r % (D / 16);
    row0 = r / (D / 16);
    d = (c >> 1) * 32 + (c & 1) * 8;
    left = int32_t(min(int64_t(p.span), p.chunks - base));
  }
  // The CTA's token of chunk j and the row within it.
  __device__ __forceinline__ void at(const Fp4CacheParams& p, int j, int& token, int& row) const {
    const uint32_t r = uint32_t(row0 + j * (kThreads / (D / 16)));
    token = int(__umulhi(r, p.magic));
    row = int(r) - token * 2 * p.heads;
  }
  __device__ __forceinline__ bool live(int j) const { return j * kThreads + int(threadIdx.x) < left; }
  __device__ __forceinline__ int tokens(const Fp4CacheParams& p) const {
    return int((int64_t(blockIdx.x) * p.span + left - 1) / p.per_token - t0) + 1;
  }
};

__device__ __forceinline__ void make_rows(const Fp4CacheParams& p, int64_t t0, Tables& tab) {
  if (int(threadIdx.x) >= 2 * p.heads) return;
  const int which = int(threadIdx.x) >= p.heads, head = threadIdx.x - which * p.heads;
  tab.row[threadIdx.x] = RowAt{static_cast<const uint8_t*>(p.rows[which]) + (t0 * p.r_s0[which] + head * p.r_s1[which]) * p.esz,
                               which * p.c_s1 + head * p.c_s2, which * p.s_s1 + head * p.s_s2};
}

template <int D>
__device__ __forceinline__ void make_tokens(const Fp4CacheParams& p, const Chunks<D>& c, Tables& tab) {
  if (int(threadIdx.x) >= c.tokens(p)) return;
  const int64_t t = c.t0 + threadIdx.x;
  int32_t page, slot;
  TokenAt at{-1, -1};
  if (page_slot(p.indptr, p.indices, p.batch, p.page_size, p.num_pages, __ldg(p.batch_indices + t),
                __ldg(p.positions + t), page, slot)) {
    at.codes = page * p.c_s0 + slot * p.c_s3;
    at.scales = page * p.s_s0 + slot * (D / kFp4Block);
  } else {
    record_error(p.st, BSKV_ERR_DEVICE_INDEX);
  }
  tab.token[threadIdx.x] = at;
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

// Largest magnitude of the two lanes' 32 values as fp32 bits; the sign-less 16-bit patterns of both
// types order as integers, a NaN above infinity.
template <typename T>
__device__ __forceinline__ uint32_t block_max(const uint4 (&x)[2]) {
  constexpr uint32_t k = 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(x[0].x & k, x[0].y & k), __vmaxu2(x[0].z & k, x[0].w & k));
  m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[1].x & k, x[1].y & k), __vmaxu2(x[1].z & k, x[1].w & k)));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m & 0xffffu, m >> 16);
  return __float_as_uint(to_float2<T>(m).x);
}

template <typename T>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = to_float2<T>(w[i]);
    packed |= cvt_e2m1x2(v.x * inv, v.y * inv) << (8 * i);
  }
  return packed;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4) fp4_append_kernel(const Fp4CacheParams p) {
  __shared__ Tables tab;
  const Chunks<D> c(p);
  make_rows(p, c.t0, tab);
  make_tokens<D>(p, c, tab);
  __syncthreads();
  for (int j0 = 0; j0 * kThreads < c.left; j0 += kUnroll) {
    uint4 x[kUnroll][2];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      int token, row;
      c.at(p, j0 + j, token, row);
      x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
      if (!c.live(j0 + j)) continue;
      const uint4* src = reinterpret_cast<const uint4*>(
          tab.row[row].rows + token * (p.r_s0[row >= p.heads] * int64_t(sizeof(T))) + c.d * sizeof(T));
      x[j][0] = __ldcs(src);
      x[j][1] = __ldcs(src + 2);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t code = e8m0_of_max(block_max<T>(x[j]));
      const float inv = e8m0_inverse(code == 255u ? 127u : code);
      const uint32_t lo = quantise8<T>(x[j][0], inv), hi = quantise8<T>(x[j][1], inv);
      if (!c.live(j0 + j)) continue;
      int token, row;
      c.at(p, j0 + j, token, row);
      const TokenAt at = tab.token[token];
      if (at.codes < 0) continue;
      const RowAt r = tab.row[row];
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + at.codes + r.codes + c.d / 2);
      dst[0] = lo;
      dst[2] = hi;
      if ((threadIdx.x & 1) == 0) p.scales[at.scales + r.scales + c.d / kFp4Block] = uint8_t(code);
    }
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
__global__ void __launch_bounds__(kThreads, 4) fp4_read_kernel(const Fp4CacheParams p) {
  __shared__ Tables tab;
  const Chunks<D> c(p);
  make_rows(p, c.t0, tab);
  make_tokens<D>(p, c, tab);
  __syncthreads();
  for (int j0 = 0; j0 * kThreads < c.left; j0 += kUnroll) {
    uint32_t w[kUnroll][2], code[kUnroll];
    T* dst[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      int token, row;
      c.at(p, j0 + j, token, row);
      dst[j] = nullptr;
      if (!c.live(j0 + j)) continue;
      const TokenAt at = tab.token[token];
      if (at.codes < 0) continue;
      const RowAt r = tab.row[row];
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.codes + at.codes + r.codes + c.d / 2);
      w[j][0] = __ldg(src);
      w[j][1] = __ldg(src + 2);
      code[j] = __ldg(p.scales + at.scales + r.scales + c.d / kFp4Block);
      dst[j] = reinterpret_cast<T*>(const_cast<uint8_t*>(r.rows) + token * (p.r_s0[row >= p.heads] * int64_t(sizeof(T)))) + c.d;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (!dst[j]) continue;
      const float f = e8m0_value(code[j]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t h[4];
        cvt_e2m1x8(w[j][half], h);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
          v[2 * i] = e.x * f;
          v[2 * i + 1] = e.y * f;
        }
        store8<T>(dst[j] + 16 * half, v);
      }
    }
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
  if (num_pages > INT32_MAX || num_kv_heads > kMaxHeads) {
    set_error("%s: num_pages=%lld num_kv_heads=%d (max %d)", who, (long long)num_pages, num_kv_heads, kMaxHeads);
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
  p->per_token = 2 * num_kv_heads * (head_dim / 16);
  p->chunks = nnz * p->per_token;
  p->esz = esz;
  p->magic = uint32_t(((uint64_t(1) << 32) + uint32_t(2 * num_kv_heads) - 1) / uint32_t(2 * num_kv_heads));
  // passes per CTA: as many as let kCtas CTAs share the input, within the token table
  const int64_t passes = (p->chunks + kPass - 1) / kPass;
  const int64_t most = std::max<int64_t>(1, int64_t(kMaxTokens - 2) * p->per_token / kPass);
  p->span = int32_t(kPass * std::min(most, (passes + kCtas - 1) / kCtas));
  if ((p->chunks + p->span - 1) / p->span > INT32_MAX) {
    set_error("%s: too many rows", who);
    return BSKV_ERR_UNSUPPORTED;
  }
  return status_args(&p->st);
}

unsigned grid_of(const Fp4CacheParams& p) { return unsigned((p.chunks + p.span - 1) / p.span); }

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
