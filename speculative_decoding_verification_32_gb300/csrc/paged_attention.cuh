// paged_attention.cuh -- parameters and device helpers shared by the kernels of
// spec_paged_attention.
//
// Keys are taken in groups of 16 tokens, a page's divisor, so a group lies in one
// page.  What a block of queries sees is one or two runs of groups: the sinks'
// (if they lie before the window) and from the group of the first token that the
// window of the block's first query reaches to that of its last token.  These
// runs are numbered through (Keys); what a query of the block does not see of
// them is masked, token by token.
//
// Sums over a part of the keys are kept as in attention.cuh:
//   m, O = sum_t 2^(x_t + e_t - m) c_t,  z = log2 sum_t 2^x_t,
// with x_t the base-2 scores, v_t = 2^e_t c_t the values (e_t = 0 and c_t = v_t
// but in a kernel that works on e4m3 codes), and parts join as
//   Z = log2 sum 2^z,  out = sum 2^(m - Z) O,  lse = ln 2 Z.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"
#include "common.cuh"
#include "kv_layout.cuh"
#include "specverify.h"

namespace sv {

constexpr int kGroup = 16;       // tokens
constexpr int kPagedSms = 152;   // items and parts are sized for this many SMs

struct PagedParams {
  const unsigned char *k, *v;  // entries
  long long page_stride, tok_stride;
  int page, pages, columns;    // tokens per page, pages in the pool, places per row
  const int32_t *table;
  const void *q;
  long long qs[3];
  float scale;                 // times log2(e)
  int B, N, Hq, H, G, D;
  const int32_t *kv_len, *count;
  int window, sinks;           // window: 0x7fffffff where every token stays visible
  // from the check kernel: each row's query count (negative: the row cannot be
  // used), and for trees the words of 32 bits of the pass's tokens that a query
  // sees, and its depth
  int32_t *rowinfo;
  int check;                   // > 0: that many of the rows kernel's first blockIdx.y make them (chains in parts)
  const uint32_t *anc;
  const int32_t *depth;
  int W;
  // partial sums: part s of output row r has O at part[at * D] and (m, z) at ml[at],
  // at = s * rows + r, and where rows are cut by a budget, so that there are no more
  // parts than run side by side, at = (item * H + KV head) * oblk + row of the block;
  // z = -inf: an empty part, O not written
  float *part;
  float2 *ml;
  int rows;                    // B * N * Hq
  int splits;                  // parts of an item's keys, at most; 1: the answers are written at once
  int budget;                  // > 0: the rows are cut into at most this many parts (cut_groups) ...
  int2 *parts_of;              // ... each into y parts, items x, x + 1, ..
  int min_groups;              // groups in a part, at least
  int oblk;                    // query rows per item
  int32_t *oflag;              // per item and part (by a budget: [item][KV head]): a value that is not finite was left out of its sums
  void *out;
  float *lse;
  int32_t *row_status;
  int qbf16;
  uint64_t wait_limit_ns;
  int force_timeout;
};

// A row's queries by its lengths alone (the check kernel looks at the rest).
__device__ __forceinline__ int paged_queries(const PagedParams &P, int b, int &n) {
  n = __ldg(P.kv_len + b);
  const int c = P.count ? __ldg(P.count + b) : P.N;
  if (n < 0 || c < 0 || c > P.N || static_cast<long long>(n) + c > static_cast<long long>(P.columns) * P.page) return kRowBadSlot;
  return c;
}

// First token that the window of a query at position p reaches.
__device__ __forceinline__ int window_from(const PagedParams &P, int p) { return p >= P.window ? p - P.window + 1 : 0; }

// The groups that queries at positions p0 .. (the first is the earliest) and
// tokens below `end` make, numbered through.
struct Keys {
  int sink, jump, n;  // groups of sinks; what is added to later numbers; groups in all
  __device__ __forceinline__ Keys(const PagedParams &P, int p0, int end) {
    const int first = window_from(P, p0) / kGroup, last = (end + kGroup - 1) / kGroup;
    sink = P.sinks / kGroup + (P.sinks % kGroup != 0);
    if (sink > first) sink = first;
    jump = first - sink;
    n = end > 0 ? last - jump : 0;
  }
  __device__ __forceinline__ int token(int i) const { return (i < sink ? i : i + jump) * kGroup; }
};

// A value of token t of row b if it is not finite, else 0.
template <int CT>
__device__ __forceinline__ float paged_odd_value(const PagedParams &P, int b, int t, int g, int d) {
  const int j = t / P.page, pg = __ldg(P.table + static_cast<size_t>(b) * P.columns + j);
  if (pg < 0 || pg >= P.pages) return 0.f;
  const unsigned char *const e = P.v + pg * P.page_stride + (t - j * P.page) * P.tok_stride;
  float val;
  if constexpr (CT == SPEC_E4M3)
    val = e[P.H * P.D + g] == 255 || (e[g * P.D + d] & 127) == 127 ? __uint_as_float(0x7fc00000u) : 0.f;
  else
    val = static_cast<float>(reinterpret_cast<const typename CacheType<CT>::type *>(e)[g * P.D + d]);
  return isfinite(val) ? 0.f : val;
}

// Whether query i of row b (at position p, n tokens before the pass) sees token t.
__device__ __forceinline__ bool paged_sees(const PagedParams &P, int b, int i, int n, int p, int t) {
  if (P.anc && t >= n) {
    const int j = t - n;
    return j < P.N && (__ldg(P.anc + (static_cast<size_t>(b) * P.N + i) * P.W + (j >> 5)) >> (j & 31) & 1u);
  }
  return t <= p && (t < P.sinks || t >= window_from(P, p));
}

// Values that are not finite, of the tokens that a query sees: its answer's
// column d gets them here, since the kernels take them out of masked groups (a
// query that does not see them would get 0 * NaN).  (Those of groups that every
// query sees went through the sums; once more changes nothing.)
template <int CT>
__device__ __noinline__ float paged_odd_sum(const PagedParams &P, int b, int i, int c, int n, int p, int g, int d) {
  float y = 0.f;
  const Keys keys(P, P.anc ? n : p, P.anc ? n + c : p + 1);  // (in a tree a sink's slot may be anywhere behind n)
  for (int k = 0; k < keys.n; ++k) {
    const int t0 = keys.token(k);
    for (int t = t0; t < t0 + kGroup; ++t)
      if (t < n + c && paged_sees(P, b, i, n, p, t)) y += paged_odd_value<CT>(P, b, t, g, d);
  }
  return y;
}

// paged_tile_kernel over all rows.
cudaError_t launch_paged_tile(const PagedParams &p, int ctype, cudaStream_t s);

}  // namespace sv
