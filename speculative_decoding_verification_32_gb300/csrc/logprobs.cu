// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives (spec_token_logprobs).
//
// With y_v = (l_v - M) log2(e) / T, M the largest logit, S = sum 2^y_v and
// U = sum y_v 2^y_v:
//   log p(v) = ln 2 (y_v - log2 S),   entropy = ln 2 (log2 S - U / S).
// (max, S, U) of two parts join by shifting to the larger max, so one pass
// over the logits is enough; its HBM read is what bounds the call.
//
// One kernel: a cluster of 1 to 8 CTAs per position (few positions are spread
// over the SMs, many take a CTA each).  A CTA runs through its slices of
// 256 x 4 16-byte vectors with the next slice's loads on their way; a thread
// takes the largest of its 32 bf16 or 16 fp32 logits (a chunk), its S and U
// against the largest so far, and leaves the chunk's maximum as a 16-bit order
// key in shared memory.  The CTAs' records join through distributed shared
// memory.  The top m are found without reading the position again: the m-th
// largest of the 256 threads' maxima is a lower bound of the m-th largest
// logit's key, and only the few chunks that reach it are looked at.  Positions
// where that leaves too many (masses of equal logits; fewer finite ones than m,
// so that -inf is among the alternatives) are searched whole by one CTA: 224
// positions of 128256 bf16 logits take 0.73 ms then, where they take 20 us.
// While one position's CTAs are at its end, others keep the memory busy: with a
// second kernel for it, 224 positions of 128256 bf16 logits took 23 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "specverify.h"

namespace sv {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpVecs = 4;  // 16-byte vectors per thread
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.442695040888963407f;
// 2^-200 is zero in fp32: stands in for the y of a masked logit, so that y 2^y is 0 and not NaN
constexpr float kFloorY = -200.f;
constexpr int kLpChunks = 1024;  // candidate chunks a CTA lists
constexpr int kLpCands = 1024;   // candidate logits it ranks
constexpr int kLpMaxCluster = 8;

struct LpPart {
  float m, s, u;
  uint32_t flags;
};

struct LpParams {
  const void *logits;
  const int32_t *tokens;
  const float *temperature;
  float *logprob, *entropy, *top_logprobs;
  int32_t *top_ids, *status;
  long long row_stride;
  int rows, npos, V, m, slice, nslices;
  int run;               // slices per CTA
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as +0
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *row, int v) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short *>(row) + v)) << 16);
  return __ldg(static_cast<const float *>(row) + v);
}

// (m, s, u) <- (m, s, u) joined with (m2, s2, u2); sc = log2(e) / T
__device__ __forceinline__ void join(float &m, float &s, float &u, float m2, float s2, float u2, float sc) {
  const float M = fmaxf(m, m2);
  if (M == -INFINITY) return;
  const float d1 = fmaxf((m - M) * sc, kFloorY), d2 = fmaxf((m2 - M) * sc, kFloorY);
  const float f1 = ex2(d1), f2 = ex2(d2);
  u = f1 * (u + d1 * s) + f2 * (u2 + d2 * s2);
  s = f1 * s + f2 * s2;
  m = M;
}

// log2(e) / T, at most kMostScale: past fp32's range (T below 2^-127) any factor puts
// every logit but the largest out of the sums, and must not make NaN of the largest.
constexpr float kMostScale = 0x1p127f;
__device__ __forceinline__ float row_temperature(const LpParams &P, int r) {
  return P.temperature ? __ldg(P.temperature + r / P.npos) : 1.f;
}
__device__ __forceinline__ float row_scale(const LpParams &P, int r, uint32_t &flags) {
  const float T = row_temperature(P, r);
  if (!(T > 0.f) || isinf(T)) {
    flags |= F_BAD_TEMPERATURE;
    return 1.f;
  }
  return fminf(kLog2e / T, kMostScale);
}
// log p of a logit d above the largest; in nats from the start (in base 2 the
// product may pass fp32's range where the result does not)
__device__ __forceinline__ float log_p(const LpParams &P, int r, float d, float sc, float lgs) {
  const float y = sc == kMostScale ? d / row_temperature(P, r) : d * (sc * kLn2);
  return y - kLn2 * lgs;
}

// One slice's logits of a thread, as they are in memory.
template <bool BF16, bool VEC>
struct LpSlice {
  static constexpr int E = BF16 ? 8 : 4;
  uint4 w[kLpVecs];

  __device__ __forceinline__ void load(const char *row, int v0, int V, int tid, uint64_t pol) {
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      const int v = v0 + (i * kLpThreads + tid) * E;
      // -inf past the end
      w[i] = BF16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                  : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
      if constexpr (VEC) {
        // V is a multiple of E here: a vector is inside or outside as a whole
        if (v < V) w[i] = ld_stream_u4(row + static_cast<size_t>(v) * (BF16 ? 2 : 4), pol);
      } else {
        uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (v + j < V) {
            if constexpr (BF16) {
              const uint32_t h = __ldg(reinterpret_cast<const unsigned short *>(row) + v + j);
              u[j / 2] = j & 1 ? (u[j / 2] & 0xffffu) | h << 16 : (u[j / 2] & 0xffff0000u) | h;
            } else {
              u[j] = __ldg(reinterpret_cast<const uint32_t *>(row) + v + j);
            }
          }
        w[i] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
  __device__ __forceinline__ float2 pair(int i, int j) const {  // elements 2 j, 2 j + 1 of vector i
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    if constexpr (BF16) return make_float2(bf16_lo(u[j]), bf16_hi(u[j]));
    return make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  }
};

// Sum over the CTA of one int per thread (all threads get it).
__device__ __forceinline__ int block_sum(int v, int *sh) {
  v = __reduce_add_sync(FULL_MASK, v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kLpThreads / 32; ++w) t += sh[w];
  return t;
}

__device__ __forceinline__ LpPart ld_remote_part(const LpPart *p, uint32_t rank) {
  const float4 v = ld_dsmem_f4(dsmem_addr(p, rank));
  return LpPart{v.x, v.y, v.z, __float_as_uint(v.w)};
}
__device__ __forceinline__ uint32_t ld_remote_u32(const void *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_remote_u64(const void *p, uint32_t rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(dsmem_addr(p, rank)) : "memory");
  return v;
}

// Grid: position * cluster size + rank (SPREAD: clusters of more than one).
// CTAs per SM as measured: 224 positions of 128256 bf16 logits 20 us at 3 and 23
// at 4 (8.4 would be the bytes at the copy rate: the rest is the end of a
// position); 2047 positions of 32000 fp32 logits 61 us at 3, 56 at 4, 54 to 56 at 5
// (4.7 TB/s, 0.69 of the copy rate; 48 registers, 32 to 96 bytes a thread spill)
// and 70 at 6, where more does.
template <bool BF16, bool VEC, bool SPREAD>
__global__ void __launch_bounds__(kLpThreads, BF16 ? 3 : 5) logprobs_kernel(const __grid_constant__ LpParams P) {
  constexpr int E = BF16 ? 8 : 4;
  __shared__ __align__(16) LpPart sh[kLpThreads / 32];
  __shared__ __align__(16) LpPart whole;        // this CTA's record
  __shared__ uint32_t tmax[kLpThreads];
  __shared__ int red[kLpThreads / 32];
  __shared__ int n_chunks, n_cands;
  __shared__ int chunk[kLpChunks];
  __shared__ unsigned long long cand[kLpCands];
  extern __shared__ __align__(16) unsigned char lp_smem[];  // this CTA's chunk keys
  unsigned short *const keys = reinterpret_cast<unsigned short *>(lp_smem);
  const uint32_t ranks = SPREAD ? cluster_nctarank() : 1u, rank = SPREAD ? cluster_ctarank() : 0u;
  const int r = blockIdx.x / ranks, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const size_t esz = BF16 ? 2 : 4;
  const char *row = static_cast<const char *>(P.logits) + static_cast<size_t>(r) * P.row_stride * esz;
  const int sl0 = rank * P.run, sl1 = min(sl0 + P.run, P.nslices);
  const int tok = P.tokens ? __ldg(P.tokens + r) : -1;
  int32_t *ids = P.top_ids + static_cast<size_t>(r) * P.m;
  float *lps = P.top_logprobs + static_cast<size_t>(r) * P.m;
  if (P.tokens && tok == -1) {  // the whole cluster leaves
    if (rank == 0) {
      for (int i = tid; i < P.m; i += kLpThreads) {
        ids[i] = -1;
        lps[i] = NAN;
      }
      if (tid == 0) {
        P.logprob[r] = NAN;
        P.entropy[r] = NAN;
        P.status[r] = 0;
      }
    }
    return;
  }
  const uint64_t pol = l2_policy_evict_normal();  // a few lines are looked at again
  LpSlice<BF16, VEC> cur, nxt;
  if (sl0 < sl1) cur.load(row, sl0 * P.slice, P.V, tid, pol);
  uint32_t flags = 0;
  const float sc = row_scale(P, r, flags);
  if (P.tokens && (tok < -1 || tok >= P.V)) flags |= F_BAD_TOKEN;
  float xt = 0.f;  // the given token's logit
  if (tok >= 0 && tok < P.V) xt = logit_at<BF16>(row, tok);
  if (tid == 0) n_chunks = n_cands = 0;
  float m = -INFINITY, s = 0.f, u = 0.f;
  uint32_t mine = 0;  // the largest of this thread's chunk keys
#pragma unroll 2  // no copies between the two slices' registers
  for (int sl = sl0; sl < sl1; ++sl) {
    if (sl + 1 < sl1) nxt.load(row, (sl + 1) * P.slice, P.V, tid, pol);
    float c = -INFINITY;  // the chunk's largest
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      if constexpr (BF16) {
        const uint32_t t = bf16x2_max_nan(bf16x2_max_nan(cur.w[i].x, cur.w[i].y), bf16x2_max_nan(cur.w[i].z, cur.w[i].w));
        c = fmax_nan(c, fmax_nan(bf16_lo(t), bf16_hi(t)));
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) c = fmax_nan(c, fmax_nan(cur.pair(i, j).x, cur.pair(i, j).y));
      }
    }
    if (!(c < INFINITY)) flags |= F_NONFINITE;  // NaN or +inf
    if (P.m > 0) {
      const uint32_t k = order_key(c) >> 16;
      keys[(sl - sl0) * kLpThreads + tid] = static_cast<unsigned short>(k);
      mine = max(mine, k);
    }
    if (c > m) {  // the sums follow the largest so far
      const float d = fmaxf((m - c) * sc, kFloorY), f = ex2(d);
      u = f * (u + d * s);
      s *= f;
      m = c;
    }
    if (m > -INFINITY) {
      const float2 sc2 = make_float2(sc, sc), off2 = make_float2(-m, -m);
      float2 s2 = make_float2(0.f, 0.f), u2 = s2;
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i)
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          float2 y = fmul2(fadd2(cur.pair(i, j), off2), sc2);
          y = make_float2(fmaxf(y.x, kFloorY), fmaxf(y.y, kFloorY));
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          s2 = fadd2(s2, e);
          u2 = ffma2(y, e, u2);
        }
      s += s2.x + s2.y;
      u += u2.x + u2.y;
    }
    cur = nxt;
  }
  // --- the position's record: threads, warps, CTAs
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join(m, s, u, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, s, o),
         __shfl_xor_sync(FULL_MASK, u, o), sc);
  flags = __reduce_or_sync(FULL_MASK, flags);
  if (lane == 0) sh[warp] = LpPart{m, s, u, flags};
  if (SPREAD) tmax[tid] = mine;
  __syncthreads();
  {
    // every warp joins the warps' records; lanes of a butterfly may round
    // differently, so one lane's result counts
    const LpPart p = lane < kLpThreads / 32 ? sh[lane] : LpPart{-INFINITY, 0.f, 0.f, 0u};
    m = p.m, s = p.s, u = p.u, flags = p.flags;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      join(m, s, u, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, s, o),
           __shfl_xor_sync(FULL_MASK, u, o), sc);
    flags = __reduce_or_sync(FULL_MASK, flags);
  }
  if constexpr (SPREAD) {
    if (tid == 0) whole = LpPart{m, s, u, flags};
    cluster_sync();
    const LpPart p = lane < static_cast<int>(ranks) ? ld_remote_part(&whole, lane) : LpPart{-INFINITY, 0.f, 0.f, 0u};
    m = p.m, s = p.s, u = p.u, flags = p.flags;
#pragma unroll
    for (int o = kLpMaxCluster / 2; o > 0; o >>= 1)
      join(m, s, u, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, s, o),
           __shfl_xor_sync(FULL_MASK, u, o), sc);
    flags = __reduce_or_sync(FULL_MASK, flags);
    for (uint32_t k = 0; k < ranks; ++k) mine = max(mine, ld_remote_u32(&tmax[tid], k));
  }
  m = __shfl_sync(FULL_MASK, m, 0);
  s = __shfl_sync(FULL_MASK, s, 0);
  u = __shfl_sync(FULL_MASK, u, 0);
  if (m == -INFINITY && !(flags & F_NONFINITE)) flags |= F_EMPTY;
  const float lgs = log2f(s);
  const bool bad = flags != 0;
  if (rank == 0 && tid == 0) {
    if (P.tokens) P.logprob[r] = bad ? NAN : log_p(P, r, xt - m, sc, lgs);
    P.entropy[r] = bad ? NAN : fmaxf(0.f, kLn2 * (lgs - u / s));
    P.status[r] = lowest_code(flags);
  }
  if (P.m == 0 || bad) {
    if (rank == 0)
      for (int i = tid; i < P.m; i += kLpThreads) {
        ids[i] = -1;
        lps[i] = NAN;
      }
    if (SPREAD) cluster_sync();  // the others may still be reading this CTA's memory
    return;
  }
  // --- a lower bound of the m-th largest chunk key: the m-th largest of the 256
  // threads' maxima, bit by bit (a barrier counts).  At least m chunks reach it,
  // and few more.  With fewer than m maxima it is 0: all are looked at.
  unsigned t16 = 0;
#pragma unroll
  for (int bit = 15; bit >= 0; --bit) {
    const unsigned t = t16 | (1u << bit);
    if (__syncthreads_count(mine >= t) >= P.m) t16 = t;
  }
  // --- this CTA's chunks that reach it, and their logits that do, a 16-byte
  // vector per thread
  for (int i = tid; i < (sl1 - sl0) * kLpThreads; i += kLpThreads)
    if (keys[i] >= t16) {
      const int at = atomicAdd(&n_chunks, 1);
      if (at < kLpChunks) chunk[at] = i;
    }
  __syncthreads();
  const int nc = n_chunks;
  for (int i = tid; i < min(nc, kLpChunks) * kLpVecs; i += kLpThreads) {
    const int c = chunk[i / kLpVecs];
    const int v0 = (sl0 + c / kLpThreads) * P.slice + ((i % kLpVecs) * kLpThreads + c % kLpThreads) * E;
    if (v0 >= P.V) continue;
    uint32_t w[4];
    if constexpr (VEC) {
      const uint4 q = __ldg(reinterpret_cast<const uint4 *>(row + v0 * esz));
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (v0 + e >= P.V) break;
      const float x = !VEC ? logit_at<BF16>(row, v0 + e) : BF16 ? (e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2])) : __uint_as_float(w[BF16 ? 0 : e]);
      const uint32_t k = order_key(x);
      if ((k >> 16) < t16) continue;
      const int at = atomicAdd(&n_cands, 1);
      if (at < kLpCands) cand[at] = static_cast<unsigned long long>(k) << 32 | (0xffffffffu - (v0 + e));
    }
  }
  __syncthreads();
  bool over = nc > kLpChunks || n_cands > kLpCands;  // too many to list
  int n = n_cands;
  if constexpr (SPREAD) {
    if (tid == 0 && over) n_cands = kLpCands + 1;
    cluster_sync();
    if (rank != 0) {
      cluster_sync();  // until rank 0 has read this CTA's list
      return;
    }
    // rank 0 appends the others' lists to its own
    for (uint32_t k = 1; k < ranks; ++k) {
      const int more = static_cast<int>(ld_remote_u32(&n_cands, k));
      over = over || more > kLpCands || n + more > kLpCands;
      if (!over)
        for (int i = tid; i < more; i += kLpThreads) cand[n + i] = ld_remote_u64(&cand[i], k);
      n += more;
    }
    cluster_sync();
  }
  if (over) {
    // Whole-position search: the m-th largest key exactly, bit by bit, then
    // everything above it (fewer than m) and the first of the equal ones.
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t tt = t | (1u << bit);
      int c = 0;
      for (int v = tid; v < P.V; v += kLpThreads) c += order_key(logit_at<BF16>(row, v)) >= tt;
      if (block_sum(c, red) >= P.m) t = tt;
    }
    if (tid == 0) n_cands = 0;
    __syncthreads();
    for (int v = tid; v < P.V; v += kLpThreads) {
      const uint32_t k = order_key(logit_at<BF16>(row, v));
      if (k > t) cand[atomicAdd(&n_cands, 1)] = static_cast<unsigned long long>(k) << 32 | (0xffffffffu - v);
    }
    __syncthreads();
    const int above = n_cands;
    int have = above;  // the same in every thread
    for (int v0 = 0; v0 < P.V && have < P.m; v0 += kLpThreads) {
      const int v = v0 + tid;
      const bool hit = v < P.V && order_key(logit_at<BF16>(row, v)) == t;
      const unsigned ball = __ballot_sync(FULL_MASK, hit);
      __syncthreads();
      if (lane == 0) red[warp] = __popc(ball);
      __syncthreads();
      int at = have, all = 0;
      for (int w = 0; w < kLpThreads / 32; ++w) {
        if (w < warp) at += red[w];
        all += red[w];
      }
      at += __popc(ball & ((1u << lane) - 1));
      if (hit && at < P.m) cand[at] = static_cast<unsigned long long>(t) << 32 | (0xffffffffu - v);
      have += all;
    }
    __syncthreads();
    n = min(have, P.m);
  }
  // rank by counting: keys are unique (the id is part of them)
  for (int i = tid; i < n; i += kLpThreads) {
    const unsigned long long k = cand[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += cand[j] > k;
    if (rank < P.m) {
      ids[rank] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(k));
      lps[rank] = log_p(P, r, from_key(static_cast<uint32_t>(k >> 32)) - m, sc, lgs);
    }
  }
}

int lp_slice(bool bf16) { return kLpThreads * kLpVecs * (bf16 ? 8 : 4); }
// CTAs per position: doubled while that leaves each a slice and the grid within
// eight per SM (384 positions of 128256 bf16 logits, 224 of them asked for: 26 us
// with one CTA each, 20 with two, 34 with four; 2047 positions of 32000 fp32
// logits: 56 us with one, 80 with two).
int lp_ranks(long long rows, int nslices) {
  int ranks = 1;
  while (ranks < kLpMaxCluster && 2 * ranks <= nslices && rows * 2 * ranks <= 8 * 152) ranks *= 2;
  return ranks;
}
bool lp_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool lp_sizes(int32_t B, int32_t npos, int32_t V) {
  return B >= 0 && npos >= 1 && V >= 1 && V <= SPEC_MAX_V && static_cast<long long>(B) * npos < 0x7fffffffLL / 64;
}

template <bool BF16, bool VEC>
cudaError_t launch_logprobs(const LpParams &p, int ranks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * ranks);
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = p.m > 0 ? static_cast<size_t>(p.run) * kLpThreads * 2 : 0;  // 32 KB at most
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  return ranks > 1 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, VEC, true>, p)
                   : cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, VEC, false>, p);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_token_logprobs(const spec_logprobs_args *a, const spec_logprobs_out *o, void *stream) {
  if (!a || !o) return SPEC_ERR_NULL;
  if (!lp_sizes(a->B, a->npos, a->V)) return SPEC_ERR_SHAPE;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (a->m < 0 || a->m > SPEC_MAX_TOP || a->m > a->V || a->row_stride < a->V) return SPEC_ERR_ARG;
  if (a->B == 0) return SPEC_OK;
  if (!a->logits || !o->entropy || !o->status || (a->tokens && !o->logprob) ||
      (a->m > 0 && (!o->top_ids || !o->top_logprobs)))
    return SPEC_ERR_NULL;
  const bool bf16 = a->dtype == SPEC_BF16;
  const int esz = bf16 ? 2 : 4;
  if (!lp_aligned(a->logits, esz)) return SPEC_ERR_ALIGN;
  const void *w4[] = {a->tokens, a->temperature, o->logprob, o->entropy, o->top_ids, o->top_logprobs, o->status};
  for (const void *q : w4)
    if (!lp_aligned(q, 4)) return SPEC_ERR_ALIGN;
  LpParams p = {};
  p.logits = a->logits;
  p.tokens = a->tokens;
  p.temperature = a->temperature;
  p.logprob = o->logprob;
  p.entropy = o->entropy;
  p.top_ids = o->top_ids;
  p.top_logprobs = o->top_logprobs;
  p.status = o->status;
  p.row_stride = a->row_stride;
  p.rows = a->B * a->npos;
  p.npos = a->npos;
  p.V = a->V;
  p.m = a->m;
  p.slice = lp_slice(bf16);
  p.nslices = (a->V + p.slice - 1) / p.slice;
  const int ranks = lp_ranks(p.rows, p.nslices);
  p.run = (p.nslices + ranks - 1) / ranks;
  const bool vec = lp_aligned(a->logits, 16) && (a->row_stride * esz) % 16 == 0 && (static_cast<long long>(a->V) * esz) % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? (vec ? launch_logprobs<true, true>(p, ranks, s) : launch_logprobs<true, false>(p, ranks, s))
                             : (vec ? launch_logprobs<false, true>(p, ranks, s) : launch_logprobs<false, false>(p, ranks, s));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
