// kv_cache.cu -- writing the verify pass's keys and values into the KV cache
// and reading entries back (spec_kv_append, spec_kv_read).
//
// Both are pure streams, bound by HBM bandwidth (or, for a handful of tokens,
// by one launch and two dependent loads).  The unit of work is 16 elements
// of one head vector in each plane: 16 e4m3 codes are one 16-byte access.
// A group of GS lanes (4 or 8, at least head_dim / 16) holds a head vector,
// so its largest magnitude is log2 GS shuffles away and nothing is read twice.
// 32768 tokens of 8 heads of 128 bf16 numbers to e4m3: 35.5 us (5.7 TB/s of
// algorithmic bytes, 0.84 of the copy rate); 32 rows of up to 2048 e4m3 entries
// read as bf16: 57 us (6.0 TB/s, 0.89).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "kv_layout.cuh"
#include "specverify.h"

namespace sv {
namespace {

// small blocks: 32768 tokens of 8 heads appended in 37.8 us at 256 threads, 35.4 at 128
constexpr int kKvcThreads = 128;

struct AppendParams {
  unsigned char *kc, *vc;
  long long row_stride, tok_stride, slots;
  const void *k, *v;
  long long ks[3], vs[3];
  const int32_t *kv_len, *count;
  int32_t *row_status;
  int rows, N, heads, D, entry;
};

// 16 elements as floats; VEC: the source is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = static_cast<float>(p[i]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldcs(reinterpret_cast<const float4 *>(p) + i);
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    }
  } else {
    uint4 u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    const T *e = reinterpret_cast<const T *>(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = static_cast<float>(e[i]);
  }
}

__device__ __forceinline__ uint4 pack_e4m3(const float (&x)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Writes one lane's 16 elements of a head vector.  `part`: which 16 of the
// vector; lanes past the vector (part >= D / 16) only take part in the
// shuffles.  The power-of-two scale makes x / s exact, so the code is the one
// rounding of the whole store (half an e4m3 step, 2^-4 relative).
template <typename T, int CT, int GS>
__device__ __forceinline__ void store16(unsigned char *e, const float (&x)[16], int h, int part, bool live,
                                        const AppendParams &P) {
  if constexpr (CT == SPEC_E4M3) {
    uint32_t a = 0;  // largest magnitude as bits: NaN > inf > finite
#pragma unroll
    for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL_MASK, a, o));
    const uint32_t c = e4m3_scale_byte(a);
    if (!live) return;
    const float inv = c == 255u ? 0.f : __uint_as_float((254u - c) << 23);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (c != 255u) w = pack_e4m3(x, inv);
    *reinterpret_cast<uint4 *>(e + h * P.D + part * 16) = w;
    const int at = P.heads * P.D + h;
    if (part == 0) e[at] = static_cast<unsigned char>(c);
    // the last head's lanes fill the entry up, so that whole sectors are written
    if (h == P.heads - 1)
      for (int i = at + 1 + part; i < P.entry; i += P.D / 16) e[i] = 0;
  } else {
    if (!live) return;
    using C = typename CacheType<CT>::type;
    alignas(16) C o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = C(x[i]);
    uint4 *to = reinterpret_cast<uint4 *>(e + 2 * (h * P.D + part * 16));
    to[0] = reinterpret_cast<const uint4 *>(o)[0];
    to[1] = reinterpret_cast<const uint4 *>(o)[1];
  }
}

// Grid: x over (token, head, lane) of one row, y = row.  The source loads do
// not wait for the row's length: they only need i < N.
template <typename T, int CT, int GS, bool VEC>
__global__ void __launch_bounds__(kKvcThreads) kv_append_kernel(const __grid_constant__ AppendParams P) {
  const int b = blockIdx.y;
  const unsigned flat = blockIdx.x * kKvcThreads + threadIdx.x;
  const unsigned g = flat / GS;
  const int part = flat % GS;
  const unsigned i = g / static_cast<unsigned>(P.heads);
  const int h = g - i * P.heads;
  const bool mine = i < static_cast<unsigned>(P.N) && part * 16 < P.D;
  const int start = __ldg(P.kv_len + b);
  const int cnt = P.count ? __ldg(P.count + b) : P.N;
  float xk[16], xv[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) xk[e] = xv[e] = 0.f;
  if (mine) {
    load16<T, VEC>(static_cast<const T *>(P.k) + b * P.ks[0] + i * P.ks[1] + h * P.ks[2] + part * 16, xk);
    load16<T, VEC>(static_cast<const T *>(P.v) + b * P.vs[0] + i * P.vs[1] + h * P.vs[2] + part * 16, xv);
  }
  const bool ok = start >= 0 && cnt >= 0 && cnt <= P.N && static_cast<long long>(start) + cnt <= P.slots;
  if (flat == 0 && P.row_status) P.row_status[b] = ok ? 0 : SPEC_ROW_BAD_SLOT;
  const bool live = mine && ok && static_cast<int>(i) < cnt;
  const long long off = b * P.row_stride + (static_cast<long long>(start) + i) * P.tok_stride;
  store16<T, CT, GS>(P.kc + off, xk, h, part, live, P);
  store16<T, CT, GS>(P.vc + off, xv, h, part, live, P);
}

struct ReadParams {
  const unsigned char *kc, *vc;
  long long row_stride, tok_stride, slots;
  void *k, *v;
  const int32_t *start, *length;
  int32_t *row_status;
  int rows, T, heads, D, entry;
};

template <typename O>
__device__ __forceinline__ void write16(O *to, const float (&x)[16]) {
  alignas(16) O o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = O(x[i]);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(O)); ++i)
    __stcs(reinterpret_cast<uint4 *>(to) + i, reinterpret_cast<const uint4 *>(o)[i]);
}

template <int CT>
__device__ __forceinline__ void read16(const unsigned char *e, int h, int part, const ReadParams &P, float (&x)[16]) {
  if constexpr (CT == SPEC_E4M3) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(e + h * P.D + part * 16));
    const float s = e4m3_scale(e[P.heads * P.D + h]);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i / 2] >> (16 * (i & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  } else {
    using C = typename CacheType<CT>::type;
    uint4 u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = __ldcs(reinterpret_cast<const uint4 *>(e + 2 * (h * P.D + part * 16)) + i);
    const C *c = reinterpret_cast<const C *>(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = static_cast<float>(c[i]);
  }
}

// Grid: x over 16-element pieces (slot t, head, part) of one row, y = row.
template <typename O, int CT>
__global__ void __launch_bounds__(kKvcThreads) kv_read_kernel(const __grid_constant__ ReadParams P) {
  const int b = blockIdx.y;
  const unsigned flat = blockIdx.x * kKvcThreads + threadIdx.x;
  const unsigned parts = P.D / 16;
  const unsigned g = flat / parts;
  const int part = flat - g * parts;
  const unsigned t = g / static_cast<unsigned>(P.heads);
  const int h = g - t * P.heads;
  const int start = P.start ? __ldg(P.start + b) : 0;
  const int len = __ldg(P.length + b);
  const bool ok = start >= 0 && len >= 0 && len <= P.T && static_cast<long long>(start) + len <= P.slots;
  if (flat == 0 && P.row_status) P.row_status[b] = ok ? 0 : SPEC_ROW_BAD_SLOT;
  if (t >= static_cast<unsigned>(P.T)) return;
  float xk[16], xv[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) xk[i] = xv[i] = 0.f;
  if (ok && static_cast<int>(t) < len) {
    const long long off = b * P.row_stride + (static_cast<long long>(start) + t) * P.tok_stride;
    read16<CT>(P.kc + off, h, part, P, xk);
    read16<CT>(P.vc + off, h, part, P, xv);
  }
  const long long at = ((static_cast<long long>(b) * P.T + t) * P.heads + h) * P.D + part * 16;
  write16(static_cast<O *>(P.k) + at, xk);
  write16(static_cast<O *>(P.v) + at, xv);
}

template <typename T, int CT, bool VEC>
void append_gs(const AppendParams &p, cudaStream_t s) {
  const int parts = p.D / 16;
  const int gs = parts <= 4 ? 4 : 8;
  const long long lanes = static_cast<long long>(p.N) * p.heads * gs;
  const dim3 grid(static_cast<unsigned>((lanes + kKvcThreads - 1) / kKvcThreads), p.rows);
  if (gs == 4)
    kv_append_kernel<T, CT, 4, VEC><<<grid, kKvcThreads, 0, s>>>(p);
  else
    kv_append_kernel<T, CT, 8, VEC><<<grid, kKvcThreads, 0, s>>>(p);
}

template <typename T>
void append_ct(const AppendParams &p, int ct, bool vec, cudaStream_t s) {
  if (ct == SPEC_E4M3)
    vec ? append_gs<T, SPEC_E4M3, true>(p, s) : append_gs<T, SPEC_E4M3, false>(p, s);
  else if (ct == SPEC_BF16)
    vec ? append_gs<T, SPEC_BF16, true>(p, s) : append_gs<T, SPEC_BF16, false>(p, s);
  else
    vec ? append_gs<T, SPEC_F16, true>(p, s) : append_gs<T, SPEC_F16, false>(p, s);
}

template <typename O>
void read_ct(const ReadParams &p, int ct, cudaStream_t s) {
  const long long pieces = static_cast<long long>(p.T) * p.heads * (p.D / 16);
  const dim3 grid(static_cast<unsigned>((pieces + kKvcThreads - 1) / kKvcThreads), p.rows);
  if (ct == SPEC_E4M3)
    kv_read_kernel<O, SPEC_E4M3><<<grid, kKvcThreads, 0, s>>>(p);
  else if (ct == SPEC_BF16)
    kv_read_kernel<O, SPEC_BF16><<<grid, kKvcThreads, 0, s>>>(p);
  else
    kv_read_kernel<O, SPEC_F16><<<grid, kKvcThreads, 0, s>>>(p);
}

bool kv_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

spec_status check_kv_cache(const spec_kv_cache &c) {
  if (c.dtype != SPEC_BF16 && c.dtype != SPEC_F16 && c.dtype != SPEC_E4M3) return SPEC_ERR_DTYPE;
  const size_t entry = spec_kv_entry_bytes(c.heads, c.head_dim, c.dtype);
  if (c.rows < 0 || c.rows > 65535 || entry == 0 || c.slots < 0 || c.slots > 0x7fffffffLL) return SPEC_ERR_SHAPE;
  if (c.row_stride < 0 || c.tok_stride < 0 || c.row_stride % 16 || c.tok_stride % 16 || !kv_aligned(c.k, 16) ||
      !kv_aligned(c.v, 16))
    return SPEC_ERR_ALIGN;
  if (c.slots > 1 && c.tok_stride < static_cast<int64_t>(entry)) return SPEC_ERR_SHAPE;
  return SPEC_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_kv_entry_bytes(int32_t heads, int32_t head_dim, int32_t dtype) {
  if (heads < 1 || heads > SPEC_MAX_HEADS || head_dim < 16 || head_dim > SPEC_MAX_HEAD_DIM || head_dim % 16) return 0;
  const size_t n = static_cast<size_t>(heads) * head_dim;
  if (dtype == SPEC_E4M3) return (n + heads + 15) / 16 * 16;
  if (dtype == SPEC_BF16 || dtype == SPEC_F16) return 2 * n;
  return 0;
}

spec_status spec_kv_append(const spec_kv_append_args *a, int32_t *row_status, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const spec_kv_cache &c = a->cache;
  if (a->src_dtype != SPEC_F32 && a->src_dtype != SPEC_BF16 && a->src_dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  const spec_status st = check_kv_cache(c);
  if (st != SPEC_OK) return st;
  if (a->N < 0 || static_cast<long long>(a->N) * c.heads * 8 > 0x7fffff00LL) return SPEC_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (a->k_stride[i] < 0 || a->v_stride[i] < 0) return SPEC_ERR_SHAPE;
  if (!kv_aligned(a->kv_len, 4) || !kv_aligned(a->count, 4) || !kv_aligned(row_status, 4)) return SPEC_ERR_ALIGN;
  if (c.rows == 0 || a->N == 0) return SPEC_OK;
  if (!c.k || !c.v || !a->k || !a->v || !a->kv_len) return SPEC_ERR_NULL;
  const int esz = a->src_dtype == SPEC_F32 ? 4 : 2;
  if (!kv_aligned(a->k, esz) || !kv_aligned(a->v, esz)) return SPEC_ERR_ALIGN;
  bool vec = kv_aligned(a->k, 16) && kv_aligned(a->v, 16);
  AppendParams p = {};
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
    vec = vec && (a->k_stride[i] * esz) % 16 == 0 && (a->v_stride[i] * esz) % 16 == 0;
  }
  p.kc = static_cast<unsigned char *>(c.k);
  p.vc = static_cast<unsigned char *>(c.v);
  p.row_stride = c.row_stride;
  p.tok_stride = c.tok_stride;
  p.slots = c.slots;
  p.k = a->k;
  p.v = a->v;
  p.kv_len = a->kv_len;
  p.count = a->count;
  p.row_status = row_status;
  p.rows = c.rows;
  p.N = a->N;
  p.heads = c.heads;
  p.D = c.head_dim;
  p.entry = static_cast<int>(spec_kv_entry_bytes(c.heads, c.head_dim, c.dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->src_dtype == SPEC_F32)
    append_ct<float>(p, c.dtype, vec, s);
  else if (a->src_dtype == SPEC_BF16)
    append_ct<__nv_bfloat16>(p, c.dtype, vec, s);
  else
    append_ct<__half>(p, c.dtype, vec, s);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_read(const spec_kv_read_args *a, int32_t *row_status, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const spec_kv_cache &c = a->cache;
  if (a->out_dtype != SPEC_F32 && a->out_dtype != SPEC_BF16 && a->out_dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  const spec_status st = check_kv_cache(c);
  if (st != SPEC_OK) return st;
  if (a->T < 0 || static_cast<long long>(a->T) * c.heads * 8 > 0x7fffff00LL) return SPEC_ERR_SHAPE;
  if (!kv_aligned(a->k_out, 16) || !kv_aligned(a->v_out, 16) || !kv_aligned(a->start, 4) ||
      !kv_aligned(a->length, 4) || !kv_aligned(row_status, 4))
    return SPEC_ERR_ALIGN;
  if (c.rows == 0 || a->T == 0) return SPEC_OK;
  if (!a->k_out || !a->v_out || !a->length || ((!c.k || !c.v) && c.slots > 0)) return SPEC_ERR_NULL;
  ReadParams p = {};
  p.kc = static_cast<const unsigned char *>(c.k);
  p.vc = static_cast<const unsigned char *>(c.v);
  p.row_stride = c.row_stride;
  p.tok_stride = c.tok_stride;
  p.slots = c.slots;
  p.k = a->k_out;
  p.v = a->v_out;
  p.start = a->start;
  p.length = a->length;
  p.row_status = row_status;
  p.rows = c.rows;
  p.T = a->T;
  p.heads = c.heads;
  p.D = c.head_dim;
  p.entry = static_cast<int>(spec_kv_entry_bytes(c.heads, c.head_dim, c.dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->out_dtype == SPEC_F32)
    read_ct<float>(p, c.dtype, s);
  else if (a->out_dtype == SPEC_BF16)
    read_ct<__nv_bfloat16>(p, c.dtype, s);
  else
    read_ct<__half>(p, c.dtype, s);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
