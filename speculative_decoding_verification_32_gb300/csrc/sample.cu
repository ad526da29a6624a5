// sample.cu -- one token per row from a truncated law at a given uniform
// (spec_sample).
//
// Every truncation is a floor on the logit: with the row's logits l, its largest
// M, w_v = exp((l_v - M) / T) and mass(t) = sum of w_v over l_v >= t,
//   top-k:  the largest t that k logits reach,
//   top-p:  the largest t with mass(t) >= top_p mass(top-k's floor),
//   min-p:  M + T ln(min_p);
// the law is w over the logits that reach all three, and the token the smallest
// v whose running sum in vocabulary order passes u times the whole.
//
// One cluster of CTAs per row.  The pass over memory finds the threads' largest
// logits and their masses against these; a slice stays in shared memory or is read
// again from L2.  The floors are found among few candidates: a bound
// below the floor that is cheap (the k-th largest of the threads' own maxima;
// for top-p some octaves below the largest weight) leaves not many more logits
// than the law keeps.  A second pass sends these to the first CTA, in vocabulary
// order, where a short list's members are held against each other and a longer
// one's floors searched bit by bit.  Where the octaves do
// not hold enough mass or too many logits, a histogram of the weights by their
// leading bits gives a nearer bound; and where more are left than the first CTA
// can list, all CTAs search together.
//
// The token is the definition's.  Sums are made of fp32 weights and rounded to
// integers (w 2^44), and every decision that hangs on one (where u falls, which side of
// top-p's border a logit is on) is held against a bound on the sums' errors (Slack).
// One that lies nearer is made again from weights in two words (exact_weight.cuh), which
// takes the row 6 us (2048 tokens) to 12 (131072, eight CTAs; 23 with two).  How often
// depends on the law: its tokens' borders, 2 slack wide each.  Of rows of 128256
// tokens drawn from whole 4% (standard deviation 3, and some tokens 9 above) and 27%
// (1), of 32000 under top-p 0.95 10%, under min-p 0.02 as well or top-k 50 0 to 0.2%.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "exact_weight.cuh"
#include "internal.h"
#include "specverify.h"

namespace sv {
namespace {

constexpr int kSmThreads = 256;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmMaxCluster = 8;
constexpr int kSmResident = 4 * 152;  // CTAs that run at a time
constexpr int kSmBatch = 8;       // 16-byte loads of a thread in flight, first pass
constexpr int kSmCands = 2048;    // candidates the first CTA lists, an equal share of them from each CTA
constexpr int kSmPairs = 256;     // ... up to so many are held against each other
constexpr int kSmPer = kSmCands / kSmThreads;
constexpr int kSmSegs = kSmWarps * kSmMaxCluster;
constexpr int kSmBins = 512;      // weights 1 down to 2^-64, eight bins an octave
constexpr float kSmFix = 0x1p44f; // a weight of 1 as an integer
constexpr float kSmMostScale = 0x1p127f;  // log2(e) / T at most: past fp32's range only the largest logit counts
constexpr uint32_t kSmMinusInf = 0x007fffffu;  // the key of -inf, the least a logit can have

struct SampleParams {
  const void *logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *token, *row_status;
  float *prob;
  long long row_stride;
  int B, V;
  int slice;    // elements per CTA, a multiple of a vector's
  int batches;  // of kSmBatch vectors, per thread
};

typedef long long i64;
typedef unsigned long long u64;

__device__ __forceinline__ uint32_t smp_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as +0
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float smp_from_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ void st_cluster_u64(const void *p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dsmem_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(const void *p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void add_cluster_u64(const void *p, uint32_t rank, u64 v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(dsmem_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void max_cluster_u32(const void *p, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(dsmem_addr(p, rank)), "r"(v) : "memory");
}
// The cluster's barrier, thread by thread: some come to it from branches of their
// own (the aligned form wants whole warps).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_meet(uint32_t ranks) {
  if (ranks == 1) {  // (the cluster's takes 1000 cycles all the same)
    __syncthreads();
    return;
  }
  cluster_arrive();
  cluster_wait();
}

struct SampleShared {
  u64 part[2][kSmMaxCluster];       // what the CTAs tell one another, two rounds in turn
  u64 part2[2][kSmMaxCluster];
  u64 warp[2][kSmWarps];            // this CTA's warps, two rounds in turn
  u64 warp2[2][kSmWarps];
  uint32_t tmax[kSmThreads];        // threads' largest keys, of the whole cluster
  unsigned char pick[kSmWarps][32]; // lanes of a batch with candidates
  uint32_t cnt[kSmSegs];            // candidates of each warp, or of each CTA
  uint32_t over[kSmMaxCluster];     // CTAs with a warp that has too many to list
  uint32_t min_p_key;
  float floor;                      // what top-p's histogram says
  uint32_t sure;                    // what was decided by fp32 weights holds
  ExactWeight exact;                // the row's weights in two words
  Words dpart[2][kSmMaxCluster];    // exact sums: of the CTAs, two in turn, and of this CTA's warps
  Words dwarp[kSmWarps];
  union {
    struct {
      u64 hist[kSmBins];            // first CTA: the cluster's
      uint32_t mine[kSmBins];       // this CTA's
    };
    u64 cand[kSmCands];             // first CTA: key << 32 | token
  };
  u64 mass[kSmPairs];               // first CTA: a short list's weights
  int at[kSmSegs];                  // ... and where its segments start
};

// Warp sum of 64-bit integers.
__device__ __forceinline__ i64 warp_sum64(i64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}
__device__ __forceinline__ i64 warp_scan64(i64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const i64 y = __shfl_up_sync(FULL_MASK, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// floor(f n) and ceil(f n) for 0 <= f < 1 and n >= 0, exactly (fp64 runs at a
// sixty-fourth of fp32's rate here, and the whole CTA would compute it).
__device__ __forceinline__ i64 fraction_of(float f, i64 n, bool up) {
  const uint32_t b = __float_as_uint(f);
  const uint32_t e = b >> 23;
  const u64 m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int s = 150 - static_cast<int>(e ? e : 1u);  // f = m 2^-s, s >= 24
  const u64 lo = m * static_cast<u64>(n), hi = __umul64hi(m, static_cast<u64>(n));
  u64 r, rest;
  if (s >= 128) {
    r = 0, rest = lo | hi;
  } else if (s >= 64) {
    r = s == 64 ? hi : hi >> (s - 64);
    rest = lo | (s == 64 ? 0 : hi << (128 - s));
  } else {
    r = hi << (64 - s) | lo >> s;
    rest = lo << (64 - s);
  }
  return static_cast<i64>(r + (up && rest ? 1 : 0));
}

// The weights of a row: w(l) = 2^((l - M) log2(e) / T), in fp32.  A weight of 2^-y is
// off by less than 3.25 ln 2 2^-24 y of itself (the difference, the product, the
// division by T, log2(e): the latter two alike for all of a row) and the hardware's
// 2^-22 for the power.  (In two words all along the passes would take ten times the
// instructions.)
struct Weight {
  float M, sc;
  __device__ __forceinline__ float operator()(float l) const { return ex2((l - M) * sc); }
  __device__ __forceinline__ float2 operator()(float2 l) const {
    const float2 y = fmul2(fadd2(l, make_float2(-M, -M)), make_float2(sc, sc));
    return make_float2(ex2(y.x), ex2(y.y));
  }
};

template <bool BF16>
__device__ __forceinline__ float element(const uint4 &q, int e) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (BF16) return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  return __uint_as_float(w[e]);
}
// The largest of a vector's logits; NaN if one is.
template <bool BF16>
__device__ __forceinline__ float vector_max(const uint4 &q) {
  if constexpr (BF16) {
    const uint32_t t = bf16x2_max_nan(bf16x2_max_nan(q.x, q.y), bf16x2_max_nan(q.z, q.w));
    return fmax_nan(bf16_lo(t), bf16_hi(t));
  }
  return fmax_nan(fmax_nan(element<BF16>(q, 0), element<BF16>(q, 1)), fmax_nan(element<BF16>(q, 2), element<BF16>(q, 3)));
}

// A vector of a row from memory; -inf past the end.
template <bool BF16, bool VEC>
__device__ __forceinline__ uint4 load_vector(const char *row, int at, int last, uint64_t policy) {
  if constexpr (VEC) {
    return ld_stream_u4(row + static_cast<size_t>(at) * (BF16 ? 2 : 4), policy);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF16) {
        const unsigned short *p = reinterpret_cast<const unsigned short *>(row) + at + 2 * e;
        w[e] = (at + 2 * e < last ? __ldg(p) : 0xff80u) | (at + 2 * e + 1 < last ? static_cast<uint32_t>(__ldg(p + 1)) : 0xff80u) << 16;
      } else {
        w[e] = at + e < last ? __ldg(reinterpret_cast<const uint32_t *>(row) + at + e) : 0xff800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// How far a sum of fp32 weights (an integer's worth) may lie from the true one, with a
// tenth to spare.  The exponents' part: sum w y <= s log2(V / s), most where all
// weights are alike.  Powers: the weight's own, the row's, and one for each time that a
// thread's largest logit grew (with every batch but the first at most).  Sums: 8
// roundings in a batch, one a batch.  And an integer's half for each vector or thread.
struct Slack {
  float V, powers;
  __device__ __forceinline__ explicit Slack(const SampleParams &P)
      : V(static_cast<float>(P.V)), powers(1.1f * ((P.batches + 1) * 0x1.4p-22f + (8 + P.batches) * 0x1p-24f)) {}
  __device__ __forceinline__ float operator()(i64 sum) const {
    const float s = fmaxf(static_cast<float>(sum) / kSmFix, 0x1p-60f);
    return (s * (1.1f * 1.35e-7f * __log2f(V / s) + powers)) * kSmFix + 0x1p16f;
  }
};

// ------------------------------------------------------------ exact decisions
// What is done for few rows stays out of line and asks for little, so that the rest
// is not slower for it.

// Dynamic shared memory: kPower32, the largest logit of every batch of vectors of every
// thread, and the slice where it is kept.
extern __shared__ __align__(16) unsigned char smp_raw[];
constexpr int kSmTable = 32 * 8;
__device__ __forceinline__ const float2 *power_table() { return reinterpret_cast<const float2 *>(smp_raw); }
__device__ __forceinline__ float *batch_largest() { return reinterpret_cast<float *>(smp_raw + kSmTable); }
__device__ __forceinline__ uint4 *kept_slice(const SampleParams &P) { return reinterpret_cast<uint4 *>(smp_raw + kSmTable + P.batches * kSmThreads * 4); }

// A CTA's part of a row, a run of vectors for each thread.
template <bool BF16, bool VEC, bool KEEP>
struct RowSlice {
  static constexpr int E = BF16 ? 8 : 4;
  const char *row;
  const uint4 *data;
  uint64_t policy;
  int first, last, vecs, per;
  __device__ __forceinline__ RowSlice(const SampleParams &P) {
    row = static_cast<const char *>(P.logits) + static_cast<size_t>(blockIdx.x / cluster_nctarank()) * P.row_stride * (BF16 ? 2 : 4);
    data = kept_slice(P);
    policy = l2_policy_evict_normal();
    first = cluster_ctarank() * P.slice;
    last = min(P.V, first + P.slice);
    vecs = last > first ? (last - first + E - 1) / E : 0;
    per = (vecs + kSmThreads - 1) / kSmThreads;
  }
  __device__ __forceinline__ uint4 operator()(int v) const { return KEEP ? data[v] : load_vector<BF16, VEC>(row, first + v * E, last, policy); }
};
__device__ __forceinline__ ExactWeight exact_weight(const SampleShared &S) {
  ExactWeight w = S.exact;
  w.power = power_table();  // (known to be shared memory)
  return w;
}

// The weights that reach `floor` in vectors from .. to - 1, by one thread.
template <bool BF16, bool VEC, bool KEEP>
__device__ __noinline__ Words lane_sum(const SampleParams &P, const SampleShared &S, float floor, int from, int to) {
  const RowSlice<BF16, VEC, KEEP> row(P);
  const ExactWeight weight = exact_weight(S);
  ExactSum<2> sum;
  uint4 q[3];  // the next ones are on their way
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (from + i < to) q[i] = row(from + i);
#pragma unroll 1
  for (int v = from; v < to; ++v) {
    if (v + 2 < to) q[2] = row(v + 2);
    if (vector_max<BF16>(q[0]) >= floor) {
#pragma unroll
      for (int e = 0; e < row.E; e += 4) {
        const float2 l[2] = {make_float2(element<BF16>(q[0], e), element<BF16>(q[0], e + 1)), make_float2(element<BF16>(q[0], e + 2), element<BF16>(q[0], e + 3))};
        float2 w[2], wl[2];
        weight(l, floor, w, wl);
        sum.add(w, wl);
      }
    }
    q[0] = q[1];
    q[1] = q[2];
  }
  return sum.all();
}

// Of the lanes' shares, one after the other from `run` on: the first that passes
// `target`, or (hit: 0) the last that is not empty; -1: all are.  What lies before it,
// and where all of them end.
struct Found {
  int lane, hit;
  Words before, end;
};
// (the first `width` lanes have some)
__device__ __noinline__ Found find_lane(Words x, int width, Words run, Words target) {
  const int lane = threadIdx.x % 32;
  if (lane >= width) x = {0.f, 0.f};
  Words inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= width) break;
    const Words y = {__shfl_up_sync(FULL_MASK, inc.hi, o), __shfl_up_sync(FULL_MASK, inc.lo, o)};
    if (lane >= o) inc = add_words(inc, y);
  }
  const Words upto = add_words(run, inc);
  const unsigned some = __ballot_sync(FULL_MASK, x.hi > 0.f), hit = some & __ballot_sync(FULL_MASK, exceeds(upto, target));
  Found f;
  f.hit = hit != 0;
  f.lane = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : -1;
  f.before = {__shfl_sync(FULL_MASK, upto.hi, max(f.lane - 1, 0)), __shfl_sync(FULL_MASK, upto.lo, max(f.lane - 1, 0))};
  if (f.lane < 1) f.before = run;
  f.end = {__shfl_sync(FULL_MASK, upto.hi, width - 1), __shfl_sync(FULL_MASK, upto.lo, width - 1)};
  return f;
}
// The shares' sum.
__device__ __forceinline__ Words sum_lanes(Words x, int width) { return find_lane(x, width, {0.f, 0.f}, {INFINITY, 0.f}).end; }

// The exact mass of the row's logits that reach `floor`, by the whole cluster, the
// same in every thread; the shares of the CTAs are in S.dpart[turn] (another one's with
// each call), of the warps in S.dwarp, and a lane's is `mine`.
template <bool BF16, bool VEC, bool KEEP>
__device__ __noinline__ Words exact_sum(const SampleParams &P, SampleShared &S, float floor, int turn, Words &mine) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ranks = cluster_nctarank();
  const RowSlice<BF16, VEC, KEEP> row(P);
  const int v = min(row.vecs, tid * row.per);
  mine = lane_sum<BF16, VEC, KEEP>(P, S, floor, v, min(row.vecs, v + row.per));
  const Words part = sum_lanes(mine, 32);
  if (lane == 0) S.dwarp[warp] = part;
  __syncthreads();
  if (warp == 0) {
    const Words all = sum_lanes(S.dwarp[lane % kSmWarps], kSmWarps);
    if (lane < static_cast<int>(ranks))
      st_cluster_u64(&S.dpart[turn][cluster_ctarank()], lane, static_cast<u64>(__float_as_uint(all.lo)) << 32 | __float_as_uint(all.hi));
  }
  cluster_meet(ranks);
  return sum_lanes(S.dpart[turn][lane % kSmMaxCluster], ranks);
}
template <bool BF16, bool VEC, bool KEEP>
__device__ __forceinline__ Words exact_mass(const SampleParams &P, SampleShared &S, float floor, int turn) {
  Words mine;
  return exact_sum<BF16, VEC, KEEP>(P, S, floor, turn, mine);
}

// The row's token from exact weights, by the whole cluster: the smallest that
// reaches `floor` and whose running sum passes u times the whole.
template <bool BF16, bool VEC, bool KEEP>
__device__ __noinline__ void draw_exact(const SampleParams &P, SampleShared &S, float floor, int turn) {
  constexpr int E = BF16 ? 8 : 4;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Words mine;
  const Words Z = exact_sum<BF16, VEC, KEEP>(P, S, floor, turn, mine);
  const int b = blockIdx.x / cluster_nctarank();
  const RowSlice<BF16, VEC, KEEP> row(P);
  const Words target = times(__ldg(P.u + b), Z);
  // (Sums made in another order round another way: where nothing passes the target, the
  // last share that is not empty has it.)
  Found f = find_lane(S.dpart[turn][lane % kSmMaxCluster], cluster_nctarank(), {0.f, 0.f}, target);
  if (f.lane != static_cast<int>(cluster_ctarank())) return;
  f = find_lane(S.dwarp[lane % kSmWarps], kSmWarps, f.before, target);
  if (f.lane != warp) return;
  f = find_lane(mine, 32, f.before, target);
  // the lane's vectors, side by side
  const int a0 = min(row.vecs, (warp * 32 + f.lane) * row.per), a1 = min(row.vecs, a0 + row.per);
  int vec = -1;
  Words run = f.before;
  for (int v = a0; v < a1; v += 32) {
    const Found g = find_lane(lane_sum<BF16, VEC, KEEP>(P, S, floor, v + lane, min(a1, v + lane + 1)), 32, run, target);
    if (g.lane >= 0) vec = v + g.lane, f = g;
    if (g.hit) break;
    run = g.end;
  }
  if (vec < 0) return;  // (only where another stream writes the row meanwhile)
  // its elements, a lane each
  const uint4 q = row(vec);
  float l = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane == e) l = element<BF16>(q, e);
  const Words x = exact_weight(S)(l, floor);
  if (lane == find_lane(x, E, f.before, target).lane) {
    P.token[b] = row.first + vec * E + lane;
    if (P.prob) P.prob[b] = x.hi / Z.hi;
    P.row_status[b] = 0;
  }
}

// Place `at` of the list of the segments one after the other.
__device__ __forceinline__ int listed_at(const SampleShared &S, int nseg, int seglen, int at) {
  int seg = 0;  // the last segment that starts at or before `at`
#pragma unroll
  for (int step = kSmSegs / 2; step > 0; step >>= 1)
    if (seg + step < nseg && S.at[seg + step] <= at) seg += step;
  return seg * seglen + at - S.at[seg];
}

// The token of a list (key 0: not in the law), by the first CTA, for u next to 0: among
// weights that an integer holds few bits of, or none.
__device__ __noinline__ void draw_small(const SampleParams &P, SampleShared &S, int b, int nseg, int seglen, int total) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const ExactWeight weight = exact_weight(S);
  // a warp's places lie side by side
  const int each = (total + kSmThreads - 1) / kSmThreads * 32, a0 = min(total, warp * each), a1 = min(total, a0 + each);
  auto weigh = [&](int at) {
    const uint32_t key = at < a1 ? static_cast<uint32_t>(S.cand[listed_at(S, nseg, seglen, at)] >> 32) : 0u;
    const float l = key ? smp_from_key(key) : -INFINITY;
    return weight(l, -INFINITY);
  };
  Words mine = {0.f, 0.f};
#pragma unroll 1
  for (int at = a0; at < a1; at += 32) mine = add_words(mine, weigh(at + lane));
  mine = sum_lanes(mine, 32);
  if (lane == 0) S.dwarp[warp] = mine;
  __syncthreads();
  const Words share = S.dwarp[lane % kSmWarps], Z = sum_lanes(share, kSmWarps), target = times(__ldg(P.u + b), Z);
  Found f = find_lane(share, kSmWarps, {0.f, 0.f}, target);
  if (f.lane != warp) return;
  int place = -1;
  float prob = 0.f;
  Words run = f.before;
#pragma unroll 1
  for (int at = a0; at < a1; at += 32) {
    const Words x = weigh(at + lane);
    f = find_lane(x, 32, run, target);
    if (f.lane == lane) place = at + lane, prob = x.hi / Z.hi;
    else if (f.lane >= 0) place = -1;
    if (f.hit) break;
    run = f.end;
  }
  if (place >= 0) {
    P.token[b] = static_cast<int>(static_cast<uint32_t>(S.cand[listed_at(S, nseg, seglen, place)]));
    if (P.prob) P.prob[b] = prob;
    P.row_status[b] = 0;
  }
}

// What a list's members are held against.
struct ListLaw {
  int nseg, seglen, total, round;  // segments, places in each, members in all; of the exchange
  int top_k;                       // 0: off
  uint32_t floor_key, top_key;     // min-p's floor, where members are not asked themselves; the largest logit's
  bool use_p, ask;
  float top_p, min_p, u, M, T;
  i64 need;                        // top-p's share of the whole row's mass (without top-k)
};

// The token of a list, by the first CTA.  By fp32 weights nothing is written, and the
// answer is true, where a decision lies nearer than their errors (open: top-p's, where
// it goes by the whole row); by exact ones (EXACT) all is decided, but for tokens
// next to u = 0.
template <bool BF16, bool EXACT>
__device__ __forceinline__ bool list_token(const SampleParams &P, SampleShared &S, int b, const ListLaw &L, const Weight &weight, const Slack &slack, float open) {
  constexpr int kLow = BF16 ? 16 : 0;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, total = L.total;
  int round = L.round;
  auto block_sum64 = [&](i64 a) {
    const int r = round & 1;
    ++round;
    a = warp_sum64(a);
    if (lane == 0) S.warp[r][warp] = static_cast<u64>(a);
    __syncthreads();
    u64 x = 0;
#pragma unroll
    for (int k = 0; k < kSmWarps; ++k) x += S.warp[r][k];
    return static_cast<i64>(x);
  };
  const int each = (total + kSmThreads - 1) / kSmThreads;  // neighbours in a thread, at most kSmPer
  uint32_t key[kSmPer];
  int id[kSmPer];
  i64 w[kSmPer];
  bool low[kSmPer];  // out by min-p
#pragma unroll
  for (int i = 0; i < kSmPer; ++i) low[i] = false, key[i] = 0, id[i] = -1, w[i] = 0;
  auto take = [&](int i) {
    const int at = tid * each + i;
    if (i < each && at < total) {
      const u64 c = S.cand[listed_at(S, L.nseg, L.seglen, at)];
      key[i] = static_cast<uint32_t>(c >> 32);
      id[i] = static_cast<int>(static_cast<uint32_t>(c));
      const float l = smp_from_key(key[i]);
      float y;
      if constexpr (EXACT) {
        const Words x = exact_weight(S)(l, -INFINITY);
        y = x.hi;
        w[i] = __float2ll_rn(y * kSmFix) + __float2ll_rn(x.lo * kSmFix);
      } else {
        y = weight(l);
        w[i] = __float2ll_rn(y * kSmFix);
      }
      // min-p: by the weight, or in fp64 where that is too near to say
      if (L.ask) {
        bool out = y < L.min_p;
        if (fabsf(y - L.min_p) <= 1e-5f * L.min_p)
          out = static_cast<double>(l) - static_cast<double>(L.M) < static_cast<double>(L.T) * log(static_cast<double>(L.min_p));
        low[i] = out;
      }
    }
  };
  take(0);
  if (each > 1) {  // (passed by at once: what is skipped piece by piece is fetched all the same)
#pragma unroll
    for (int i = 1; i < kSmPer; ++i) take(i);
  }
  bool unsure = false;
  i64 need = L.need;
  if (total <= kSmPairs) {
    // --- few: each thread holds its candidate (each = 1) against all of them
    if (tid < total) S.mass[tid] = static_cast<u64>(w[0]), S.tmax[tid] = key[0];
    __syncthreads();
    i64 above = 0;
    int larger = 0;
    if (tid < total)
#pragma unroll 4
      for (int j = 0; j < total; ++j) {
        const bool gt = S.tmax[j] > key[0];
        larger += gt;
        above += gt ? static_cast<i64>(S.mass[j]) : 0;
      }
    bool keep = tid < total && key[0] >= L.floor_key && !low[0] && (!L.top_k || larger < L.top_k);
    if (L.top_k && L.use_p) {
      const i64 mass = block_sum64(tid < total && larger < L.top_k ? w[0] : 0);
      need = fraction_of(L.top_p, mass, true);
      open = 2.f * slack(mass);
    }
    if (L.use_p) {
      if (!EXACT) unsure = keep && fabsf(static_cast<float>(above - need)) <= open;
      keep = keep && above < need;
    }
    if (!keep) w[0] = 0, id[0] = -1;
  } else {
    uint32_t floor = L.floor_key, least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kSmPer; ++i)
      if (id[i] >= 0) least = min(least, key[i]);
    {
      const int r = round & 1;
      ++round;
      least = __reduce_min_sync(FULL_MASK, least);
      if (lane == 0) S.warp[r][warp] = least;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSmWarps; ++k) least = min(least, static_cast<uint32_t>(S.warp[r][k]));
    }
    if (L.top_k) {
      uint32_t lo = least >> kLow, hi = L.top_key >> kLow;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        int n = 0;
#pragma unroll
        for (int i = 0; i < kSmPer; ++i) n += id[i] >= 0 && key[i] >= mid << kLow;
        if (block_sum64(n) >= L.top_k) lo = mid;
        else hi = mid - 1;
      }
      floor = max(floor, lo << kLow);
      if (L.use_p) {
        i64 a = 0;
#pragma unroll
        for (int i = 0; i < kSmPer; ++i)
          if (key[i] >= lo << kLow) a += w[i];
        a = block_sum64(a);
        need = fraction_of(L.top_p, a, true);
        open = 2.f * slack(a);
        least = max(least, lo << kLow);
      }
    }
    if (L.use_p) {
      uint32_t lo = least >> kLow, hi = L.top_key >> kLow;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        i64 a = 0;
#pragma unroll
        for (int i = 0; i < kSmPer; ++i)
          if (key[i] >= mid << kLow) a += w[i];
        a = block_sum64(a);
        if (!EXACT) unsure = unsure || fabsf(static_cast<float>(a - need)) <= open;
        if (a >= need) lo = mid;
        else hi = mid - 1;
      }
      floor = max(floor, lo << kLow);
    }
#pragma unroll
    for (int i = 0; i < kSmPer; ++i)
      if (key[i] < floor || low[i]) w[i] = 0, id[i] = -1;
  }
  // --- running sums in vocabulary order
  i64 mine = 0;
#pragma unroll
  for (int i = 0; i < kSmPer; ++i) mine += w[i];
  const i64 inc = warp_scan64(mine, lane);
  const int r = round & 1;
  if (lane == 31) S.warp[r][warp] = static_cast<u64>(inc);
  unsure = __syncthreads_or(unsure);
  if (unsure) return true;
  i64 run = inc - mine, all = 0;
#pragma unroll
  for (int k = 0; k < kSmWarps; ++k) {
    const i64 x = static_cast<i64>(S.warp[r][k]);
    if (k < warp) run += x;
    all += x;
  }
  const i64 target = fraction_of(L.u, all, false);
  if (EXACT && target < 1 << 20) {
#pragma unroll
    for (int i = 0; i < kSmPer; ++i)
      if (id[i] < 0 && i < each && tid * each + i < total) S.cand[listed_at(S, L.nseg, L.seglen, tid * each + i)] = 0;
    __syncthreads();
    draw_small(P, S, b, L.nseg, L.seglen, total);
    return false;
  }
  int token = -1;
  i64 its = 0, low_end = 0;
#pragma unroll
  for (int i = 0; i < kSmPer; ++i) {
    if (run <= target && run + w[i] > target) token = id[i], its = w[i], low_end = run;
    run += w[i];
  }
  bool sure = false;
  if (token >= 0) {
    const float off = slack(all);
    sure = EXACT || (static_cast<float>(target - low_end) > off && static_cast<float>(low_end + its - target) > off);
    if (sure) {
      P.token[b] = token;
      if (P.prob) P.prob[b] = static_cast<float>(its) / static_cast<float>(all);
      P.row_status[b] = 0;
    }
  }
  return EXACT ? false : !__syncthreads_or(sure);
}
template <bool BF16, bool VEC, bool KEEP>
__device__ __noinline__ void list_token_exact(const SampleParams &P, SampleShared &S, int b, const ListLaw &law) {
  ListLaw L = law;
  if (L.use_p && !L.top_k) {
    const Words share = times(L.top_p, exact_mass<BF16, VEC, KEEP>(P, S, -INFINITY, 0));
    L.need = max(1LL, __float2ll_rn(share.hi * kSmFix) + __float2ll_ru(share.lo * kSmFix));  // (the largest logits stay)
  }
  __syncthreads();  // (the exchange's buffers start anew)
  list_token<BF16, true>(P, S, b, L, Weight{L.M, 0.f}, Slack(P), 0.f);
}

// KEEP: slices stay in shared memory; else later passes read them again, from L2.
template <bool BF16, bool VEC, bool KEEP>
__global__ void __launch_bounds__(kSmThreads, 4) sample_kernel(const __grid_constant__ SampleParams P) {
  constexpr int E = BF16 ? 8 : 4;
  __shared__ SampleShared S;
  float *const largest = batch_largest();
  uint4 *const data = kept_slice(P);
  const uint32_t ranks = cluster_nctarank(), rank = cluster_ctarank();
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const char *row = static_cast<const char *>(P.logits) + static_cast<size_t>(b) * P.row_stride * (BF16 ? 2 : 4);
  const int first = rank * P.slice, last = min(P.V, first + P.slice);  // may be empty
  const int vecs = last > first ? (last - first + E - 1) / E : 0;
  // a warp's vectors lie side by side, so that warps and lanes are in vocabulary order
  const int per = (vecs + 32 * kSmWarps - 1) / (32 * kSmWarps) * 32;
  const int v0 = min(vecs, warp * per), v1 = min(vecs, v0 + per);

  S.tmax[tid] = 0;
  if (tid < 32) reinterpret_cast<float2 *>(smp_raw)[tid] = kPower32[tid];
  if (tid == 0) S.sure = 0;
  cluster_arrive();  // the others must be running before anything is stored into their memory
  // --- the slice, and its largest logit
  const uint64_t policy = KEEP ? l2_policy_evict_first() : l2_policy_evict_normal();
  auto vector_at = [&](int v) { return KEEP ? data[v] : load_vector<BF16, VEC>(row, first + v * E, last, policy); };
  const float T = P.temperature ? __ldg(P.temperature + b) : 1.f, u = __ldg(P.u + b);
  const int k_raw = P.top_k ? __ldg(P.top_k + b) : 0;
  const int top_k = k_raw >= 1 && k_raw < P.V ? k_raw : 0;  // 0: off
  const float top_p = P.top_p ? __ldg(P.top_p + b) : 1.f, min_p = P.min_p ? __ldg(P.min_p + b) : 0.f;
  const bool use_p = top_p > 0.f && top_p < 1.f, use_m = min_p > 0.f && min_p <= 1.f;
  Weight weight;
  weight.sc = fminf(1.4426950408889634f / T, kSmMostScale);
  uint32_t flags = 0;
  float top = -INFINITY, mass = 0.f;  // sum of the weights against the thread's largest so far
  int chunk = 0;
  for (int i0 = v0 + lane; i0 < v1; i0 += 32 * kSmBatch, ++chunk) {
    uint4 q[kSmBatch];
#pragma unroll
    for (int i = 0; i < kSmBatch; ++i) {
      const int v = i0 + i * 32;
      q[i] = BF16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                  : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
      if (v < v1) q[i] = load_vector<BF16, VEC>(row, first + v * E, last, policy);
    }
    float c = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSmBatch; ++i) {
      const int v = i0 + i * 32;
      if (KEEP && v < v1) data[v] = q[i];
      c = fmax_nan(c, vector_max<BF16>(q[i]));
    }
    largest[chunk * kSmThreads + tid] = c;
    if (!(c < INFINITY)) flags |= F_NONFINITE;  // NaN or +inf
    if (c > top) {
      mass *= ex2((top - c) * weight.sc);
      top = c;
    }
    if (top > -INFINITY) {
      weight.M = top;
      float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kSmBatch; ++i) {
        auto pair = [&](int e) { return weight(make_float2(element<BF16>(q[i], e), element<BF16>(q[i], e + 1))); };
        float2 x = fadd2(pair(0), pair(2));
        if constexpr (BF16) x = fadd2(x, fadd2(pair(4), pair(6)));
        s[i % 2] = fadd2(s[i % 2], x);
      }
      s[0] = fadd2(s[0], s[1]);
      mass += s[0].x + s[0].y;
    }
  }
  const uint32_t my_top = smp_key(top);
  {
    const uint32_t k = __reduce_max_sync(FULL_MASK, my_top);
    flags = __reduce_or_sync(FULL_MASK, flags);
    if (lane == 0) S.warp[0][warp] = static_cast<u64>(k) << 32 | flags;
  }
  __syncthreads();
  cluster_wait();
  {
    u64 k = 0;
    uint32_t f = 0;
#pragma unroll
    for (int w = 0; w < kSmWarps; ++w) {
      k = max(k, S.warp[0][w] >> 32);
      f |= static_cast<uint32_t>(S.warp[0][w]);
    }
    if (tid < static_cast<int>(ranks)) st_cluster_u64(&S.part[0][rank], tid, k << 32 | f);
  }
  // (every CTA's columns have been cleared: it has arrived)
  if (top_k && top_k <= kSmThreads)
    for (uint32_t k = 0; k < ranks; ++k) max_cluster_u32(&S.tmax[tid], k, my_top);
  cluster_meet(ranks);
  uint32_t top_key = 0;
  flags = 0;
  for (uint32_t k = 0; k < ranks; ++k) {
    top_key = max(top_key, static_cast<uint32_t>(S.part[0][k] >> 32));
    flags |= static_cast<uint32_t>(S.part[0][k]);
  }
  const float M = smp_from_key(top_key);
  // --- the row's numbers
  if (!(T > 0.f) || isinf(T)) flags |= F_BAD_TEMPERATURE;
  if (!(u >= 0.f && u < 1.f)) flags |= F_BAD_UNIFORM;
  if (M == -INFINITY && !(flags & F_NONFINITE)) flags |= F_EMPTY;
  if (flags) {  // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      P.token[b] = -1;
      if (P.prob) P.prob[b] = NAN;
      P.row_status[b] = lowest_code(flags);
    }
    return;
  }
  weight.M = M;
  if (tid == kSmThreads - 1) S.exact = ExactWeight(M, T, power_table());  // (800 cycles, which whoever needs it would wait for)
  // temperatures whose reciprocals or differences leave fp32's range: exact weights alone
  const bool far = !(T >= 0x1p-64f && T <= 0x1p64f);
  const Slack slack(P);
  // min-p's floor in fp32, put below it by more than what that rounds
  const float min_p_low = use_m ? M + log2f(min_p) / weight.sc - (1e-5f - 1e-5f * log2f(min_p)) / weight.sc - 0x1p-21f * fabsf(M) : -INFINITY;

  // a vector's sum of the weights that reach `floor`, as an integer
  auto vector_mass = [&](const uint4 &q, float floor) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 l = make_float2(element<BF16>(q, e), element<BF16>(q, e + 1)), w = weight(l);
      s = fadd2(s, make_float2(l.x >= floor ? w.x : 0.f, l.y >= floor ? w.y : 0.f));
    }
    return __float2ll_rn((s.x + s.y) * kSmFix);
  };
  int round = 1;  // of the exchange: buffers in turn
  // sums over the cluster (two at a time), the same in every thread
  auto exchange = [&](i64 a, i64 c, i64 &A, i64 &C) {
    const int r = round & 1;
    ++round;
    a = warp_sum64(a);
    c = warp_sum64(c);
    if (lane == 0) S.warp[r][warp] = static_cast<u64>(a), S.warp2[r][warp] = static_cast<u64>(c);
    __syncthreads();
    if (tid < static_cast<int>(ranks)) {
      u64 x = 0, y = 0;
#pragma unroll
      for (int w = 0; w < kSmWarps; ++w) x += S.warp[r][w], y += S.warp2[r][w];
      st_cluster_u64(&S.part[r][rank], tid, x);
      st_cluster_u64(&S.part2[r][rank], tid, y);
    }
    cluster_meet(ranks);
    A = C = 0;
    for (uint32_t k = 0; k < ranks; ++k) A += static_cast<i64>(S.part[r][k]), C += static_cast<i64>(S.part2[r][k]);
    return r;
  };
  // mass and count of what reaches the key
  auto reach = [&](uint32_t key, i64 &mass, i64 &count) {
    const float floor = smp_from_key(key);
    i64 a = 0;
    int n = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
      const uint4 q = vector_at(v);
      if (!(vector_max<BF16>(q) >= floor)) continue;
      a += vector_mass(q, floor);
#pragma unroll
      for (int e = 0; e < E; ++e) n += element<BF16>(q, e) >= floor;
    }
    return exchange(a, n, mass, count);
  };
  // The token at u: all CTAs together, from the sums that exchange number r left.
  // A running sum of integers passes u Z where it passes floor(u Z).  Nothing is
  // written, and S.sure left 0, where the sums' errors leave the token open.
  auto choose = [&](float floor, int r, i64 Z) {
    const i64 target = fraction_of(u, Z, false);  // less than Z, so it is passed
    int owner = 0;
    i64 before = 0;
    for (uint32_t k = 0; k < ranks; ++k) {
      const i64 x = static_cast<i64>(S.part[r][k]);
      if (before + x > target) break;
      before += x;
      ++owner;
    }
    if (owner != static_cast<int>(rank)) return;
    int w = 0;
    for (; w < kSmWarps; ++w) {
      const i64 x = static_cast<i64>(S.warp[r][w]);
      if (before + x > target) break;
      before += x;
    }
    const i64 start = before;
    // that warp's part of the slice, an eighth to each warp
    const int lo = min(vecs, w * per), hi = min(vecs, lo + per), each = (per / 32 + kSmWarps - 1) / kSmWarps * 32;
    const int a0 = min(hi, lo + warp * each), a1 = min(hi, a0 + each);
    i64 sum = 0;
    for (int i0 = a0 + lane; i0 < a1; i0 += 32 * 4) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i * 32 < a1) q[i] = vector_at(i0 + i * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i * 32 < a1) sum += vector_mass(q[i], floor);
    }
    sum = warp_sum64(sum);
    if (lane == 0) S.warp2[r][warp] = static_cast<u64>(sum);
    __syncthreads();
    int part = -1;
    for (int k = 0; k < kSmWarps; ++k) {
      const i64 x = static_cast<i64>(S.warp2[r][k]);
      if (x == 0) continue;
      if (part >= 0) before += static_cast<i64>(S.warp2[r][part]);
      part = k;
      if (before + x > target) break;
    }
    if (part != warp) return;
    for (int v = a0; v < a1; v += 32) {
      const int mine = v + lane;
      uint4 q = make_uint4(0, 0, 0, 0);
      i64 x = 0;
      if (mine < a1) {
        q = vector_at(mine);
        x = vector_mass(q, floor);
      }
      const i64 inc = warp_scan64(x, lane);
      const unsigned hit = __ballot_sync(FULL_MASK, before + inc > target);
      if (!hit) {
        before += __shfl_sync(FULL_MASK, inc, 31);
        continue;
      }
      if (lane == __ffs(hit) - 1) {  // its sums up to each element
        const i64 base = before + inc - x;
        float s = 0.f, prob = 0.f;
        i64 low = base, high = base;
        int tok = -1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float l = element<BF16>(q, e), y = l >= floor ? weight(l) : 0.f;
          s += y;
          if (high <= target && y > 0.f) {
            tok = first + mine * E + e;
            prob = y;
            low = high;
            high = base + __float2ll_rn(s * kSmFix);
          }
        }
        // The token is right if low (1 - u) <= u (Z - low) and high (1 - u) > u (Z - high)
        // for the true sums.  (What lies behind the token is the whole less what lies
        // before it, of which the warp's own part has been added up twice.)
        const float below = (1.f - u) * slack(low) + u * (slack(Z - low) + 2.f * slack(low - start));
        const float above = (1.f - u) * slack(high) + u * (slack(Z - high) + 2.f * slack(high - start));
        if (tok >= 0 && static_cast<float>(target - low) > below && static_cast<float>(high - target) > above) {
          P.token[b] = tok;
          if (P.prob) P.prob[b] = prob * kSmFix / static_cast<float>(Z);
          P.row_status[b] = 0;
          for (uint32_t k = 0; k < ranks; ++k) st_cluster_u32(&S.sure, k, 1);
        }
      }
      return;
    }
  };
  // the token by fp32 weights, and where these leave it open by exact ones
  int turn = 0;
  auto draw = [&](float floor, int r, i64 Z) {
    if (!far) {
      choose(floor, r, Z);
      cluster_meet(ranks);
      if (S.sure) return;
    }
    draw_exact<BF16, VEC, KEEP>(P, S, floor, turn);
  };

  // --- a bound that the law's floor does not lie below: the k-th largest of the
  // 256 columns' maxima, to 16 bits; min-p's floor; and for top-p some octaves
  // below the largest weight, which holds if the mass within them, found in the
  // same pass, is enough.  (Where top-p goes by the mass that top-k leaves, what
  // reaches top-k's floor has to be listed whole.)
  const bool near = use_p && !top_k && !far;
  const float near_floor = near ? M - (5.f - log2f(1.f - top_p)) / weight.sc : -INFINITY;
  float from = top_k && use_p ? -INFINITY : fmaxf(min_p_low, near_floor);
  if (top_k && top_k <= kSmThreads) {
    uint32_t mine[kSmThreads / 32], least = 0xffffu;
#pragma unroll
    for (int i = 0; i < kSmThreads / 32; ++i) least = min(least, mine[i] = S.tmax[i * 32 + lane] >> 16);
    least = __reduce_min_sync(FULL_MASK, least);
    // all of them reach the least; the bits below those that all have in common
    const uint32_t apart = least ^ (top_key >> 16);
    int bit = apart ? 31 - __clz(apart) : -1;
    uint32_t t = bit < 0 ? least : least >> (bit + 1) << (bit + 1);
#pragma unroll 1
    for (; bit >= 0; --bit) {
      const uint32_t x = t | 1u << bit;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kSmThreads / 32; ++i) n += mine[i] >= x;
      if (static_cast<int>(__reduce_add_sync(FULL_MASK, n)) >= top_k) t = x;
    }
    from = fmaxf(from, smp_from_key(max(t << 16, kSmMinusInf)));
  }
  const bool plain = !top_k && !use_p && !use_m, bounded = from > -INFINITY && !far;
  // --- the logits from the bound on into the first CTA's list, warp by warp and so
  // in vocabulary order; and the row's mass
  int nseg = kSmWarps * ranks, seglen = kSmCands / nseg;
  i64 Z, within;
  {
    const int seg = rank * kSmWarps + warp;
    const bool count_near = near && from == near_floor;
    const i64 a = top > -INFINITY ? __float2ll_rn(mass * ex2((top - M) * weight.sc) * kSmFix) : 0;
    float c = 0.f;
    int n = 0;
    // Only the vectors of lanes whose batch holds one are looked at, and by all lanes:
    // 2^width such lanes' first, second, ... vectors side by side, so that the lanes
    // are in vocabulary order and a batch with up to four is read at once.  (Each lane
    // looking at its own: three trips to L2 a batch, 256 rows 32 us, so 25.)
    for (int i0 = v0, turn = 0; i0 < v1 && bounded; i0 += 32 * kSmBatch, ++turn) {
      const bool here = i0 + lane < v1 && largest[turn * kSmThreads + tid] >= from;
      const unsigned those = __ballot_sync(FULL_MASK, here);
      if (!those) continue;
      const int found = __popc(those), width = found <= 4 ? 2 : 32 - __clz(found - 1);
      if (here) S.pick[warp][__popc(those & ((1u << lane) - 1u))] = static_cast<unsigned char>(lane);
      __syncwarp();
      const int r = lane & ((1 << width) - 1), step = 32 >> width;
      const int col = r < found ? S.pick[warp][r] : 0;
      __syncwarp();
      int v = i0 + (lane >> width) * 32 + col;
      uint4 next = make_uint4(0, 0, 0, 0);
      if (r < found && v < v1) next = vector_at(v);
#pragma unroll 1
      for (int j = 0; j < kSmBatch; j += step) {
        const uint4 q = next;
        const int mine = v;
        v += step * 32;
        if (j + step < kSmBatch && r < found && v < v1) next = vector_at(v);
        uint32_t bits = 0;
        if (r < found && mine < v1) {
#pragma unroll
          for (int e = 0; e < E; ++e) bits |= element<BF16>(q, e) >= from ? 1u << e : 0u;
        }
        const unsigned some = __ballot_sync(FULL_MASK, bits != 0);
        if (!some) continue;
        int to, all;  // the lane's first place, and places for the warp
        if (__any_sync(FULL_MASK, bits & (bits - 1))) {
          const int hits = __popc(bits);
          int inc = hits;
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += y;
          }
          to = n + inc - hits;
          all = __shfl_sync(FULL_MASK, inc, 31);
        } else {
          to = n + __popc(some & ((1u << lane) - 1u));
          all = __popc(some);
        }
        n += all;
        while (bits) {
          const int e = __ffs(bits) - 1;
          bits &= bits - 1;
          const int word = BF16 ? e >> 1 : e;
          uint32_t x = word & 2 ? (word & 1 ? q.w : q.z) : (word & 1 ? q.y : q.x);
          if (BF16) x = e & 1 ? x & 0xffff0000u : x << 16;
          const float l = __uint_as_float(x);
          if (count_near) c += ex2((l - M) * weight.sc);
          if (n <= seglen) st_cluster_u64(&S.cand[seg * seglen + to++], 0, static_cast<u64>(smp_key(l)) << 32 | static_cast<uint32_t>(first + mine * E + e));
        }
      }
    }
    if (lane == 0) st_cluster_u32(&S.cnt[seg], 0, n);
    const bool many = __syncthreads_or(n > seglen);
    if (tid < static_cast<int>(ranks)) st_cluster_u32(&S.over[rank], tid, many);
    // (the second sum is a bound: cut by more than its rounding)
    const int r = exchange(a, __float2ll_rn(c * (kSmFix * (1.f - 0x1p-14f))), Z, within);
    if (plain) {
      draw(-INFINITY, r, Z);
      return;
    }
    if (!count_near) within = Z;  // the bound holds as it is
  }
  const i64 want = use_p ? fraction_of(top_p, Z, true) : 0;  // of the whole row's mass
  // ... and a share of it that is more than top-p's, whatever the sums' errors
  const i64 ample = use_p ? want + static_cast<i64>(2.f * slack(Z)) : 0;
  bool listed = bounded && within >= ample;
  for (uint32_t k = 0; k < ranks; ++k) listed = listed && !S.over[k];
  uint32_t floor_key = kSmMinusInf;  // min-p's, where the list's members are not asked themselves
  bool ask = use_m;
  uint32_t bound = smp_key(far ? -INFINITY : near && within < ample ? min_p_low : from);
  if (!listed) {
    ask = false;
    // min-p's floor: the least logit with l - M >= T ln(min_p)
    if (tid == 0) {
      uint32_t k = kSmMinusInf;
      if (use_m) {
        const double below = static_cast<double>(T) * log(static_cast<double>(min_p)), at = static_cast<double>(M) + below;
        k = smp_key(at < -3.4028234e38 ? -3.4028234e38f : static_cast<float>(at));
        while (static_cast<double>(smp_from_key(k)) - static_cast<double>(M) < below) ++k;
        while (k > 0x00800000u && static_cast<double>(smp_from_key(k - 1)) - static_cast<double>(M) >= below) --k;
      }
      S.min_p_key = k;
    }
    cluster_meet(ranks);  // (the list is read by no one, and may be written over)
    floor_key = S.min_p_key;
    if (!(top_k && use_p)) bound = max(bound, floor_key);
  }
  bool binned = !near;
  const int share = kSmCands / static_cast<int>(ranks);
  if (!listed) {
    // --- where the law keeps much, or top-p's mass reaches far down
    if (!binned) {
      binned = true;
      for (int i = tid; i < kSmBins; i += kSmThreads) S.hist[i] = 0, S.mine[i] = 0;
      cluster_meet(ranks);
      // What is dropped weighs less than (1 - top_p) Z, so a token of less than a
      // V-th of that cannot be the last one kept: such tokens are not looked at.
      const float least = (1.f - top_p) * 0.999f * (static_cast<float>(Z) / kSmFix) / P.V;
      const float far = M + (log2f(fmaxf(least, 1e-37f)) - 0.01f) / weight.sc;
      from = fmaxf(far, smp_from_key(bound));
      // Bins by exponent and three more bits of the weight; each adds up the
      // leading 16 bits of its weights, cut off: never too much.
      for (int v = v0 + lane; v < v1; v += 32) {
        const uint4 q = vector_at(v);
        if (!(vector_max<BF16>(q) >= from)) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float l = element<BF16>(q, e);
          if (l >= from) {
            const uint32_t x = __float_as_uint(fminf(weight(l), 1.f));
            const int bin = (127 << 3) - static_cast<int>(x >> 20);
            if (bin < kSmBins) atomicAdd(&S.mine[bin], ((x & 0x7fffffu) | 0x800000u) >> 8);
          }
        }
      }
      __syncthreads();  // (a slice has at most 2^16 logits: its sums stay below 2^32)
      for (int i = tid; i < kSmBins; i += kSmThreads)
        if (S.mine[i]) add_cluster_u64(&S.hist[i], 0, S.mine[i]);
      cluster_meet(ranks);
      if (rank == 0) {
        // running sums from the largest weights down, in the sums' unit; bin i
        // holds weights of exponent -ceil(i / 8), 16 bits of each
        const int i0 = 2 * tid;
        i64 x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int s = 44 - 15 - (i0 + j + 7) / 8;
          x[j] = static_cast<i64>(s >= 0 ? S.hist[i0 + j] << s : -s < 64 ? S.hist[i0 + j] >> -s : 0);
        }
        const i64 inc = warp_scan64(x[0] + x[1], lane);
        const int r = round & 1;
        if (lane == 31) S.warp[r][warp] = static_cast<u64>(inc);
        if (tid == 0) S.floor = from;
        __syncthreads();
        i64 run = inc - x[0] - x[1];
        for (int w = 0; w < warp; ++w) run += static_cast<i64>(S.warp[r][w]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (run < ample && run + x[j] >= ample)  // one bin only: its least weight, as a logit
            S.floor = fmaxf(from, M + (log2f(__uint_as_float(static_cast<uint32_t>((127 << 3) - i0 - j) << 20)) - 0.001f) / weight.sc);
          run += x[j];
        }
        __syncthreads();
        if (tid > 0 && tid < static_cast<int>(ranks)) st_cluster_u32(&S.floor, tid, __float_as_uint(S.floor));
      }
      ++round;
      cluster_meet(ranks);
      bound = max(bound, smp_key(S.floor));
    }
    // --- the candidates, in vocabulary order
    from = smp_from_key(bound);
    int n = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
      const uint4 q = vector_at(v);
      if (!(vector_max<BF16>(q) >= from)) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) n += element<BF16>(q, e) >= from;
    }
    n = __reduce_add_sync(FULL_MASK, n);
    const int r = round & 1;
    ++round;
    if (lane == 0) S.warp[r][warp] = n;
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSmWarps; ++w) {
      const int x = static_cast<int>(S.warp[r][w]);
      if (w < warp) at += x;
      all += x;
    }
    if (tid < static_cast<int>(ranks)) st_cluster_u32(&S.cnt[rank], tid, all);
    if (all <= share && n > 0) {
      for (int v = v0; v < v1; v += 32) {
        const int mine = v + lane;
        uint4 q = make_uint4(0, 0, 0, 0);
        int c = 0;
        if (mine < v1) {
          q = vector_at(mine);
          if (vector_max<BF16>(q) >= from) {
#pragma unroll
            for (int e = 0; e < E; ++e) c += element<BF16>(q, e) >= from;
          }
        }
        if (!__any_sync(FULL_MASK, c > 0)) continue;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULL_MASK, inc, o);
          if (lane >= o) inc += y;
        }
        int to = at + inc - c;
        if (c > 0) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float l = element<BF16>(q, e);
            // (the bound on `to` holds even if another stream is writing the row meanwhile)
            if (l >= from && to < share) st_cluster_u64(&S.cand[rank * share + to++], 0, static_cast<u64>(smp_key(l)) << 32 | static_cast<uint32_t>(first + mine * E + e));
          }
        }
        at += __shfl_sync(FULL_MASK, inc, 31);
      }
    }
    cluster_meet(ranks);
    listed = true;
    for (uint32_t k = 0; k < ranks; ++k) listed = listed && static_cast<int>(S.cnt[k]) <= share;
    nseg = ranks, seglen = share;
  }
  constexpr int kLow = BF16 ? 16 : 0;  // a bf16 logit's key is its upper 16 bits
  if (!listed) {
    // --- too many: the floors by bisection, all CTAs together.  (In units of
    // 2^kLow; a key's lower bits are ones for negative numbers, so the unit's
    // first key reaches what the unit's logit does.)
    i64 mass = 0, count = 0, need = want;
    uint32_t floor = floor_key;
    float of = -INFINITY, open = use_p ? top_p * slack(Z) : 0.f;  // whose share is needed, and how far that may be off
    if (top_k) {
      uint32_t lo = bound >> kLow, hi = top_key >> kLow;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        reach(mid << kLow, mass, count);
        if (count >= top_k) lo = mid;
        else hi = mid - 1;
      }
      floor = max(floor_key, lo << kLow);
      if (use_p) {
        of = smp_from_key(max(lo << kLow, kSmMinusInf));
        reach(max(lo << kLow, kSmMinusInf), mass, count);
        need = fraction_of(top_p, mass, true);
        open = top_p * slack(mass);
        bound = max(bound, lo << kLow);
      }
    }
    if (use_p) {
      // Of sets whose mass is too near to say, by their sizes (each holds the smaller ones):
      // the smallest that is known to be enough, the largest that is known not to be.
      Words whole = {-1.f, 0.f};
      i64 ample_n = 1LL << 40, short_n = -1;
      uint32_t lo = bound >> kLow, hi = top_key >> kLow;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        reach(mid << kLow, mass, count);
        bool enough = mass >= need;
        if (far || fabsf(static_cast<float>(mass - need)) <= open + slack(mass)) {
          if (count < ample_n && count > short_n) {
            if (whole.hi < 0.f) whole = exact_mass<BF16, VEC, KEEP>(P, S, of, turn), turn ^= 1;
            if (exceeds(times(top_p, whole), exact_mass<BF16, VEC, KEEP>(P, S, smp_from_key(mid << kLow), turn))) short_n = count;
            else ample_n = count;
            turn ^= 1;
          }
          enough = count >= ample_n;
        }
        if (enough) lo = mid;
        else hi = mid - 1;
      }
      floor = max(floor, lo << kLow);
    }
    const int r = reach(floor, mass, count);
    draw(smp_from_key(floor), r, mass);
    return;
  }
  // top-p's border goes by the whole row's mass: where fp32 weights leave something open,
  // by the exact one, to which all CTAs add their part
  const bool whole_row = use_p && !top_k;
  if (rank != 0) {
    if (whole_row) {
      cluster_meet(ranks);
      if (!S.sure) exact_mass<BF16, VEC, KEEP>(P, S, -INFINITY, 0);
    }
    return;
  }
  // the list's segments, one after the other
  int total = 0;
  {
    // two counts a lane, their running sums, in every warp
    const int c0 = 2 * lane < nseg ? static_cast<int>(S.cnt[2 * lane]) : 0, c1 = 2 * lane + 1 < nseg ? static_cast<int>(S.cnt[2 * lane + 1]) : 0;
    int inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL_MASK, inc, o);
      if (lane >= o) inc += y;
    }
    total = __shfl_sync(FULL_MASK, inc, 31);
    if (warp == 0) S.at[2 * lane] = inc - c0 - c1, S.at[2 * lane + 1] = inc - c1;
  }
  __syncthreads();
  const ListLaw law = {nseg, seglen, total, round, top_k, floor_key, top_key, use_p, ask, top_p, min_p, u, M, T, want};
  bool unsure = far;
  // (both sides of the comparison may be off)
  if (!far) unsure = list_token<BF16, false>(P, S, b, law, weight, slack, whole_row ? 2.f * slack(Z) : 0.f);
  if (whole_row) {
    if (tid < static_cast<int>(ranks)) st_cluster_u32(&S.sure, tid, !unsure);
    cluster_meet(ranks);
  }
  if (unsure) list_token_exact<BF16, VEC, KEEP>(P, S, b, law);
}

bool smp_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Dynamic shared memory above 48 KB has to be asked for, once per device.
template <bool BF16, bool VEC, bool KEEP>
cudaError_t launch_sample(const SampleParams &p, int ranks, cudaStream_t s) {
  if (KEEP) {
    static std::atomic<uint64_t> done{0};
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(done.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(sample_kernel<BF16, VEC, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, 144 << 10);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * ranks);
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = kSmTable + static_cast<size_t>(p.batches) * kSmThreads * 4 + (KEEP ? static_cast<size_t>(p.slice) * (BF16 ? 2 : 4) : 0);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<BF16, VEC, KEEP>, p);
}
template <bool BF16, bool VEC>
cudaError_t launch_sample(const SampleParams &p, int ranks, bool keep, cudaStream_t s) {
  return keep ? launch_sample<BF16, VEC, true>(p, ranks, s) : launch_sample<BF16, VEC, false>(p, ranks, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_sample(const spec_sample_args *a, const spec_sample_out *o, void *stream) {
  if (!a || !o) return SPEC_ERR_NULL;
  if (a->B < 0 || a->B > 0x7fffffff / 64 || a->V < 1 || a->V > SPEC_MAX_V) return SPEC_ERR_SHAPE;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (a->row_stride < a->V) return SPEC_ERR_ARG;
  if (a->B == 0) return SPEC_OK;
  if (!a->logits || !a->u || !o->token || !o->row_status) return SPEC_ERR_NULL;
  const bool bf16 = a->dtype == SPEC_BF16;
  const int esz = bf16 ? 2 : 4;
  if (!smp_aligned(a->logits, esz)) return SPEC_ERR_ALIGN;
  const void *w4[] = {a->u, a->temperature, a->top_k, a->top_p, a->min_p, o->token, o->prob, o->row_status};
  for (const void *q : w4)
    if (!smp_aligned(q, 4)) return SPEC_ERR_ALIGN;
  SampleParams p = {};
  p.logits = a->logits;
  p.u = a->u;
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.token = o->token;
  p.prob = o->prob;
  p.row_status = o->row_status;
  p.row_stride = a->row_stride;
  p.B = a->B;
  p.V = a->V;
  // CTAs per row: slices of at most 32 KB, as far as eight go.  They stay in shared memory
  // where they all run at once: with three quarters of what the SMs' memory has room
  // for, since clusters of eight leave some of it.  Else slices are read again from L2,
  // which holds what runs at a time, and more rows than run side by side so are cut into
  // fewer slices: of 2^16 logits at most (256 rows of 128256 under top-p and min-p 26 us,
  // with 2^15 32), and of 2^15 where there is no truncation, since some of many rows'
  // sums have to be made again (256 rows of bf16 45 us, with 2^16 53; 300 of fp32 63 and
  // 77).  Kept and read again, us: 19 rows of 128256 fp32
  // logits under min-p 11.7 and 11.8, searched under top-p 0.9 181 and 209; 38 rows
  // 15.8 and 12.8, 297 and 253; 19 of 200000 16.7 and 12.4, 386 and 310; of bf16 38 rows
  // 12.2 and 12.0, 97 and 114; 76 16.2 and 14.5, 147 and 174.
  const long long bytes = static_cast<long long>(a->V) * esz;
  int ranks = 1;
  while (ranks < kSmMaxCluster && bytes > ranks * (32LL << 10)) ranks *= 2;
  const long long cta = sizeof(SampleShared) + kSmTable + 4096 + (bytes + ranks - 1) / ranks;  // its shared memory, about
  const bool keep = static_cast<long long>(a->B) * ranks * 4 <= 152 * std::min(4LL, (227LL << 10) / cta) * 3;
  if (!keep) {
    const int most = a->top_k || a->top_p || a->min_p ? 1 << 16 : 1 << 15;
    while (ranks > 1 && static_cast<long long>(a->B) * ranks > kSmResident && (a->V + ranks / 2 - 1) / (ranks / 2) <= most) ranks /= 2;
  }
  const int unit = 16 / esz;
  p.slice = ((a->V + ranks - 1) / ranks + unit - 1) / unit * unit;
  // (a warp's vectors are whole rows of 32, as in the kernel)
  const int turns = (p.slice / unit + 32 * kSmWarps - 1) / (32 * kSmWarps);
  p.batches = (turns + kSmBatch - 1) / kSmBatch;
  const bool vec = smp_aligned(a->logits, 16) && (a->row_stride * esz) % 16 == 0 && bytes % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? (vec ? launch_sample<true, true>(p, ranks, keep, s) : launch_sample<true, false>(p, ranks, keep, s))
                             : (vec ? launch_sample<false, true>(p, ranks, keep, s) : launch_sample<false, false>(p, ranks, keep, s));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
