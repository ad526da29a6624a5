// attention.cuh -- parameters and small device helpers shared by the kernels
// of spec_prefix_attention.
//
// For a query row (row b, token i, query head h) let x_t = scale log2(e) q.k_t
// be its base-2 scores and v_t = 2^e_t c_t the values of token t (e_t = 0 and
// c_t = v_t in a 16-bit cache; in an e4m3 cache c_t are the codes and 2^e_t the
// scale).  A part of the keys is summed up as
//   m = max_t (x_t + e_t),  O = sum_t 2^(x_t + e_t - m) c_t,  z = log2 sum_t 2^x_t,
// (m may lie below that: weights of the codes then reach 2^8, in the tile kernel
// 2^15.5) so the weights of the codes stay in range, whatever the scales, and the
// query's answer over several parts is
//   Z = log2 sum 2^z,  out = sum 2^(m - Z) O,  lse = ln 2 Z.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "kv_layout.cuh"
#include "specverify.h"

namespace sv {

struct AttnParams {
  // caches
  const unsigned char *k, *v;    // own entries
  const unsigned char *pk, *pv;  // prefix entries
  // the prefix of an e4m3 cache as fp16 (attn_widen_kernel), or NULL: keys then
  // values, [P][H][D]; and per head and 128 tokens the keys' scale, then the
  // values' scale exponent
  unsigned char *wide;
  float *wide_scale;
  int32_t *wide_far;  // ... whether the block's scales lie too far apart for fp16
  long long row_stride, tok_stride, ptok_stride, slots;
  int P;  // prefix length
  // queries
  const void *q;
  long long qs[3];
  float scale;  // times log2(e)
  int B, N, Hq, H, G, D;
  const int32_t *kv_len, *count;
  // tree: words of 32 ancestor bits per query (node i's own bit among them)
  // and each row's query count (negative: bad row), from the mask kernel
  const uint32_t *anc;
  const int32_t *rowinfo;
  int W;
  // partial sums: slot s of output row r has O at part[(s * rows + r) * D] and
  // (m, z) at ml[s * rows + r]; z = -inf: an empty part, O not written
  float *part;
  float2 *ml;
  int rows;         // B * N * Hq
  int psplits, pchunk;  // prefix parts (slots 0 .. psplits - 1) and tokens in each
  int osplits;          // own parts (slots psplits ..)
  int chunk, min_chunk; // own parts: multiples of `chunk` tokens, `min_chunk` at least
  int budget;           // > 0: the rows are cut into at most this many parts (cut_rows) ...
  int32_t *nparts;      // ... each into this many (else osplits)
  int oblk;             // query rows per own item
  int32_t *oflag;       // per own item: a value that is not finite was left out of its sums
  // outputs
  void *out;
  float *lse;
  int32_t *row_status;
  int qbf16;
  int first;   // the tile kernel is the first of its kind in the call
  int next;    // the rows kernel follows the prefix's tile kernel: started while that one ends
  int fuse;    // own items of the tile kernel take the prefix too
  int direct;  // ... and write the answers themselves: there is nothing to join
  uint64_t wait_limit_ns;
  int force_timeout;  // 1: every item; 2 + g: those of KV head g
};

constexpr int kRowBadSlot = -1, kRowBadParent = -2;
// z of a part whose kernel gave up waiting (no arithmetic makes this NaN)
constexpr uint32_t kTimeoutBits = 0x7fc0deadu;

// Queries of row b; negative if the row cannot be used.
__device__ __forceinline__ int row_queries(const AttnParams &P, int b) {
  if (P.rowinfo) return __ldg(P.rowinfo + b);
  const int n = __ldg(P.kv_len + b), c = P.count ? __ldg(P.count + b) : P.N;
  if (n < 0 || c < 0 || c > P.N || static_cast<long long>(n) + c > P.slots) return kRowBadSlot;
  return c;
}

// How a few rows of any lengths are cut into at most `budget` parts that can all
// run side by side, none much longer than another (the lanes of a warp together):
// item `idx` is part `split` of row `b`, tokens t0 .. t1 - 1.  A lane keeps rows
// 4 lane .. 4 lane + 3.  Lengths count in blocks of 16 tokens (w); a row makes
// max(1, ceil(w / c)) parts of c blocks, and c is the shortest length, searched
// upwards from sum w / budget, at which the budget holds: it does for
// c = sum w / (budget - B) + 1, since sum ceil(w / c) <= sum w / c + B.
constexpr int kKeep = 4;
constexpr int kMaxCutRows = 32 * kKeep;
// ceil(w / c) for w < 2^24: the quotient by a reciprocal, put right by one
__device__ __forceinline__ uint32_t ceil_quotient(uint32_t w, uint32_t c, float inv) {
  uint32_t q = static_cast<uint32_t>(static_cast<float>(w) * inv);
  if (q * c >= w + c) --q;  // one too many
  return q + (q * c < w);
}
__device__ __forceinline__ void cut_rows(const AttnParams &P, int idx, int &b, int &split, int &parts, int &t0, int &t1) {
  const int lane = threadIdx.x % 32;
  uint32_t w[kKeep], sum = 0, top = 0;
#pragma unroll
  for (int q = 0; q < kKeep; ++q) {
    const int r = lane * kKeep + q;
    w[q] = 0;
    if (r < P.B) {
      const int c = row_queries(P, r);
      if (c > 0) w[q] = static_cast<uint32_t>(__ldg(P.kv_len + r) + c + 15) / 16;  // < 2^24 blocks (checked by the caller)
    }
    sum += w[q];
    top = max(top, w[q]);
  }
  sum = __reduce_add_sync(FULL_MASK, sum);
  top = __reduce_max_sync(FULL_MASK, top);
  const uint32_t least = max((top + P.osplits - 1) / P.osplits, static_cast<uint32_t>(P.min_chunk / 16));
  const uint32_t most = sum / (P.budget - P.B) + 1;
  uint32_t c = sum / P.budget + 1, n[kKeep], mine;
  while (true) {
    c = max(min(c, most), least);
    mine = 0;
    const float inv = 1.f / static_cast<float>(c);
#pragma unroll
    for (int q = 0; q < kKeep; ++q) {
      n[q] = lane * kKeep + q < P.B ? max(1u, ceil_quotient(w[q], c, inv)) : 0u;
      mine += n[q];
    }
    if (c >= most || __reduce_add_sync(FULL_MASK, mine) <= static_cast<uint32_t>(P.budget)) break;
    c += c / 16 + 1;
  }
  // the row of item idx: inclusive sums over the lanes
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL_MASK, upto, o);
    if (lane >= o) upto += y;
  }
  const uint32_t from = upto - mine;
  const unsigned owner = __ballot_sync(FULL_MASK, static_cast<uint32_t>(idx) >= from && static_cast<uint32_t>(idx) < upto);
  b = -1;
  if (!owner) return;  // past the last part
  uint32_t k = idx - from;
  int row = lane * kKeep, cnt = 0, blocks = 0;
#pragma unroll
  for (int q = 0; q < kKeep; ++q) {
    if (q < kKeep - 1 && row == lane * kKeep + q && k >= n[q]) {
      k -= n[q];
      ++row;
    } else if (row == lane * kKeep + q) {
      cnt = static_cast<int>(n[q]);
      blocks = static_cast<int>(w[q]);
    }
  }
  const int src = __ffs(owner) - 1;
  b = __shfl_sync(FULL_MASK, row, src);
  split = __shfl_sync(FULL_MASK, static_cast<int>(k), src);
  parts = __shfl_sync(FULL_MASK, cnt, src);
  blocks = __shfl_sync(FULL_MASK, blocks, src);
  t0 = min(split * static_cast<int>(c), blocks) * 16;
  t1 = min(t0 + static_cast<int>(c) * 16, blocks * 16);  // the last part's end is the row's, which the caller knows
}

// The own part `split` covers of a row's len entries: equal parts, rounded up
// to P.chunk tokens (a power of two), none shorter than P.min_chunk but the last.
__device__ __forceinline__ void own_range(const AttnParams &P, int len, int split, int &t0, int &t1) {
  int chunk = (len + P.osplits - 1) / P.osplits;
  chunk = max(P.min_chunk, (chunk + P.chunk - 1) & -P.chunk);
  const long long a = static_cast<long long>(split) * chunk;
  t0 = static_cast<int>(min(a, static_cast<long long>(len)));
  t1 = static_cast<int>(min(a + chunk, static_cast<long long>(len)));
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two floats rounded to a pair of the 16-bit type, lo in the low half
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two e4m3 codes (the low 16 bits) as a pair of fp16: exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Exponent of a scale byte as a float; 255 (NaN) has none, and its callers give it one.
__device__ __forceinline__ float scale_exponent(uint32_t c) { return static_cast<float>(static_cast<int>(c) - 127); }
// sum_t 2^(x_t - m) is kept as l 2^-E, E the largest scale exponent met so far
// (at least kMinExponent), so that it stays in range for scales this near; a token
// whose scale is more than 2^kExponentSpan below the largest counts with that
// span and takes the rest of the factor on its weight.  That is right for the
// least scales (bytes up to kLeastScale, 2^-120: zero vectors), whose weight is
// nothing; where others lie that far apart, the kernels go other ways.
constexpr float kMinExponent = -60.f;
constexpr float kExponentSpan = 60.f;
constexpr uint32_t kLeastScale = 7;
constexpr float kLn2 = 0.693147180559945309f;

// A value of row b's own entry in slot t if it is not finite, else 0.
template <int CT>
__device__ __forceinline__ float odd_value(const AttnParams &P, int b, int t, int g, int d) {
  const unsigned char *const e = P.v + b * P.row_stride + t * P.tok_stride;
  float val;
  if constexpr (CT == SPEC_E4M3)
    val = e[P.H * P.D + g] == 255 || (e[g * P.D + d] & 127) == 127 ? __uint_as_float(0x7fc00000u) : 0.f;
  else
    val = static_cast<float>(reinterpret_cast<const typename CacheType<CT>::type *>(e)[g * P.D + d]);
  return isfinite(val) ? 0.f : val;
}

// A query's element.
__device__ __forceinline__ float query_value(unsigned short u, int bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

// A query's sums over tokens p0 .. p1 - 1 of the prefix and t0 .. t1 - 1 of its row's
// own e4m3 entries from the codes, in fp32, by one thread: for parts in which
// scales lie further apart than the kernels' ways span (a token that nothing
// sees, or whose weight is nothing, must not cost the others their bits).
// Not met by scales within 2^15 of one another, and slower by up to three and a half
// orders: with one prefix token's values 2^40 up, 32 trees of 60 nodes behind 4097
// tokens (the answers' items hold prefix and own entries) take 0.70 s where they take
// 0.20 ms without; 64 decoding rows behind 8192, parts of four blocks, 42 ms where
// they take 0.077, and 4.7 ms with such a token in every row's own entries instead.
// len0: own entries that every query sees; my, anc: the query's index and
// ancestor bits; qoff: where it is; odd: values of the pass's own tokens that
// are not finite are to be put into an answer that is written here (P.direct).
__device__ __forceinline__ void exact_part(const AttnParams &P, int b, int g, int p0, int p1, int t0, int t1, int len0, int cnt, int my,
                                           const uint32_t *anc, bool use, long long qoff, long long orow, int slot, bool odd) {
  const unsigned short *const q = static_cast<const unsigned short *>(P.q) + qoff;
  float m = -INFINITY, top = -INFINITY, l = 0.f, z = -INFINITY;
  // the first round: maxima and the sum of the softmax; then 32 columns a round
#pragma unroll 1
  for (int d0 = -32; d0 < P.D; d0 += 32) {
    float o[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = 0.f;
#pragma unroll 1
    for (int part = 0; use && part < 2; ++part) {
      const bool pre = part == 0;
      const int end = pre ? p1 : t1;
      const long long ts = pre ? P.ptok_stride : P.tok_stride;
      const unsigned char *const kb = pre ? P.pk : P.k + b * P.row_stride, *const vb = pre ? P.pv : P.v + b * P.row_stride;
#pragma unroll 1
      for (int t = pre ? p0 : t0; t < end; ++t) {
        const int own = pre ? -1 : t - len0;  // index among the pass's own tokens
        if (own >= 0 && !(anc ? __ldg(anc + (own >> 5)) >> (own & 31) & 1u : own <= my)) continue;
        const unsigned char *const ke = kb + t * ts, *const ve = vb + t * ts;
        float x = 0.f;
#pragma unroll 1
        for (int d = 0; d < P.D; d += 16) {
          const uint4 w = __ldg(reinterpret_cast<const uint4 *>(ke + static_cast<long long>(g) * P.D + d));
          const uint32_t cw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t h = e & 1 ? e4m3x2_to_f16x2_hi(cw[e / 2]) : e4m3x2_to_f16x2(cw[e / 2]);
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x = fmaf(query_value(q[d + 2 * e], P.qbf16), y.x, x);
            x = fmaf(query_value(q[d + 2 * e + 1], P.qbf16), y.y, x);
          }
        }
        x = x * e4m3_scale(__ldg(ke + static_cast<long long>(P.H) * P.D + g)) * P.scale;
        const uint32_t vc = __ldg(ve + static_cast<long long>(P.H) * P.D + g);
        const float xe = x + (vc == 255u ? 0.f : scale_exponent(vc));
        if (d0 < 0) {
          m = fmaxf(m, xe);
          if (x > top) {
            l *= ex2(top - x);
            top = x;
          }
          l += x == -INFINITY ? 0.f : ex2(x - top);
          continue;
        }
        const float w = ex2(xe - m);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (d0 + c * 16 >= P.D) continue;
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(ve + static_cast<long long>(g) * P.D + d0 + c * 16));
          const uint32_t cw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t h = e & 1 ? e4m3x2_to_f16x2_hi(cw[e / 2]) : e4m3x2_to_f16x2(cw[e / 2]);
            float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            if (vc == 255u) y.x = y.y = __uint_as_float(0x7fc00000u);
            if (own >= 0) {  // put into the answers at the end, as in every part
              if (!isfinite(y.x)) y.x = 0.f;
              if (!isfinite(y.y)) y.y = 0.f;
            }
            o[c * 16 + 2 * e] = fmaf(w, y.x, o[c * 16 + 2 * e]);
            o[c * 16 + 2 * e + 1] = fmaf(w, y.y, o[c * 16 + 2 * e + 1]);
          }
        }
      }
    }
    const bool some = use && l != 0.f;
    if (d0 < 0) {
      z = some ? top + log2f(l) : -INFINITY;
      if (!P.direct)
        P.ml[static_cast<long long>(slot) * P.rows + orow] = some ? make_float2(m, z) : make_float2(-INFINITY, -INFINITY);
      else if (P.lse)
        P.lse[orow] = kLn2 * z;
      continue;
    }
    if (P.direct) {
      const float w = some ? ex2(m - z) : 0.f;
      unsigned short *const to = static_cast<unsigned short *>(P.out) + orow * P.D + d0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (d0 + j >= P.D) continue;
        float y = some ? o[j] * w : 0.f;
        if (some && odd)
          for (int t = 0; t < cnt; ++t)
            if (anc ? __ldg(anc + (t >> 5)) >> (t & 31) & 1u : t <= my) y += odd_value<SPEC_E4M3>(P, b, len0 + t, g, d0 + j);
        to[j] = static_cast<unsigned short>(P.qbf16 ? pack16<true>(y, 0.f) : pack16<false>(y, 0.f));
      }
    } else if (some) {
      float *const to = P.part + (static_cast<long long>(slot) * P.rows + orow) * P.D + d0;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (d0 + j < P.D) to[j] = o[j];
    }
  }
}

// 32 bytes, a whole sector, aligned to 32
__device__ __forceinline__ void st_global_v8(float *p, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Raises a kernel's dynamic shared memory limit, once per device.  A kernel
// whose roles trade registers must have been given `regs` of them at launch
// (else the roles that take more would wait for ever): checked here.
template <auto Kernel>
cudaError_t allow_smem(int bytes, int regs = 0) {
  static std::atomic<uint64_t> done{0};
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  if (regs) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, Kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs != regs) return cudaErrorInvalidConfiguration;
  }
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may start before the kernel ahead of it in the stream is over
// (`early`; it then waits for that one itself, grid_dependency_wait).
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, bool early, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Host launchers.
// attn_rows_kernel over the own entries (own) and the prefix (prefix).
cudaError_t launch_attn_rows(const AttnParams &p, int ctype, bool prefix, cudaStream_t s);
// The prefix of an e4m3 cache into P.wide; runs beside the mask kernel, if there is one.
cudaError_t launch_attn_widen(const AttnParams &p, cudaStream_t s);
// attn_tile_kernel over the prefix, or over the own entries.
cudaError_t launch_attn_tile(const AttnParams &p, int ctype, bool prefix, cudaStream_t s);

}  // namespace sv
