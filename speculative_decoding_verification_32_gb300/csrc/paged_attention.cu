// paged_attention.cu -- attention over a paged cache with a sliding window and
// first tokens that stay visible (spec_paged_attention): the entry point, the
// check of the rows, the kernel for few query rows and the join of the parts.
//
//  paged_check_kernel -- one CTA per row: lengths, the pages that the row needs,
//    and for draft trees the parents, each node's depth and which of the pass's
//    tokens it sees.  The attention kernel runs beside it and looks at the
//    result before it writes anything.  (Chains in parts: a few warps of the rows
//    kernel do this, and the join looks.)
//  paged_tile_kernel (paged_attention_tile.cu) -- many query rows.
//  paged_rows_kernel -- 8 to 32 query rows (the query heads of one KV head and
//    tokens of one row) against a part of their keys, one warp.
//  paged_join_kernel -- one warp per query row adds up the parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "paged_attention.cuh"

namespace sv {
namespace {

constexpr float kPaLazy = 8.f;
constexpr float kLog2e = 1.442695040888963407f;
constexpr int kCheckThreads = 256;
constexpr int kPaJoinThreads = 128;
// Rows of more tokens are not cut by a budget: cut_groups counts groups of 16 of them
// in fp32 and adds up 128 rows' in 32 bits.  (What its own few queries bring may be above.)
constexpr long long kMaxCutTokens = (1LL << 28) - 4096;

// -------------------------------------------------------------- row check
// Whether every page that the row's queries see is there: by `threads` threads, of
// which this is the `t`-th.
__device__ __forceinline__ bool pages_there(const PagedParams &P, int b, int n, int c, int t, int threads) {
  bool paged = true;
  if (c > 0) {  // the pages of what the row's first query and later ones see
    const Keys keys(P, n, n + c);
    const int per = P.page / kGroup, row = keys.n;
    for (int k = t; k < row; k += threads) {
      const int g = keys.token(k) / kGroup;
      if (k > 0 && k != keys.sink && g % per) continue;  // the page of the group before
      const int pg = __ldg(P.table + static_cast<size_t>(b) * P.columns + g / per);
      paged = paged && pg >= 0 && pg < P.pages;
    }
  }
  return paged;
}

__global__ void __launch_bounds__(kCheckThreads) paged_check_kernel(const __grid_constant__ PagedParams P, const int32_t *parent,
                                                                    uint32_t *anc, int32_t *depth) {
  __shared__ int par[SPEC_MAX_TREE_NODES];
  const int b = blockIdx.x, tid = threadIdx.x;
  allow_dependents();
  int n;
  const int c = paged_queries(P, b, n);
  bool tree = true;
  const int used = parent ? max(0, min(P.count ? P.count[b] : P.N, P.N)) : 0;
  for (int i = tid; i < used; i += kCheckThreads) {
    const int p = parent[static_cast<size_t>(b) * P.N + i];
    par[i] = p;
    tree = tree && (i == 0 ? p == -1 : p >= 0 && p < i);
  }
  bool paged = pages_there(P, b, n, c, tid, kCheckThreads);
  tree = __syncthreads_and(tree);
  paged = __syncthreads_and(paged);
  const int code = !tree ? kRowBadParent : !paged || c < 0 ? kRowBadSlot : c;
  if (tid == 0) {
    P.rowinfo[b] = code;
    if (P.row_status) P.row_status[b] = code >= 0 ? 0 : code == kRowBadParent ? SPEC_ROW_BAD_PARENT : SPEC_ROW_BAD_SLOT;
  }
  if (code < 0) return;
  for (int i = tid; i < used; i += kCheckThreads) {
    int d = 0;
    for (int j = par[i]; j >= 0; j = par[j]) ++d;
    depth[static_cast<size_t>(b) * P.N + i] = d;
    // ancestors within the window, or sinks themselves, from the node up
    uint32_t *const row = anc + (static_cast<size_t>(b) * P.N + i) * P.W;
    int w = P.W - 1, back = 0;
    uint32_t bits = 0;
    for (int j = i; j >= 0; j = par[j], ++back) {  // indexes fall strictly on the way up
      while (w > (j >> 5)) {
        row[w--] = bits;
        bits = 0;
      }
      if (back < P.window || n + d - back < P.sinks) bits |= 1u << (j & 31);
    }
    while (w >= 0) {
      row[w--] = bits;
      bits = 0;
    }
  }
}

// ------------------------------------------------------------- row kernel
// The products are made the other way round: scores as K Q^T, sums as V^T P^T, so
// that keys fill the matrix instruction's 16 rows and query rows go in eights: 4
// rows of a decoding token are padded to 8, 24 of a chain not at all.  (With the
// queries as the 16 rows every item does twice to 4/3 of the work, with the
// registers of twice the sums: 64 decoding rows of 4 in e4m3 100 us, this way 84; 64
// chains of 24 rows 132 and 103, in bf16 105 and 97.  It is the better way for
// just 16 rows over codes alone, 60 and 68 us for 32 rows.)
template <int CT, int DP, int NT>
struct PagedRowCfg {
  static constexpr bool E4 = CT == SPEC_E4M3;
  static constexpr int kEsz = E4 ? 1 : 2;
  static constexpr int kM = 8 * NT;                         // query rows
  static constexpr int kStages = 2;                         // (64 decoding rows in e4m3 3 us more with three)
  static constexpr int kPitch = DP * kEsz + 16;             // bytes of one token in a ring slot
  static constexpr int kPlane = kGroup * kPitch;            // K or V of a group
  static constexpr int kScales = E4 ? 2 * kGroup * 4 : 0;   // scale words, K then V
  static constexpr int kStage = 2 * kPlane + kScales;
  static constexpr int kQPitch = DP * 2 + 16;
  static constexpr int kQ = kM * kQPitch + kM * 4;          // queries and factors, in the last slot before it is used, or by themselves
  static constexpr int kOPitch = DP + 4;                    // floats: eight rows of sums at the end
  // 32 rows' queries stay in shared memory, behind the ring, and are not held in
  // registers: these do not take their fragments beside the sums (64 chains of 8 over
  // codes 174 us, so 133; bf16 116 and 109; 24 rows' fit: no difference).  16 rows' over
  // codes make room for 12 items (32 decoding rows of 16 73 us, so 68; 24 rows' sums
  // would spill then: 107 and 145).
  static constexpr bool kHeld = E4 ? NT % 2 == 1 : NT <= 3;
  static constexpr int kQAt = (kHeld ? kStages - 1 : kStages) * kStage;
  static constexpr int kLast = kHeld && kStage > kQ ? kStages * kStage : kQAt + kQ;
  static constexpr int kSmem = kLast > 8 * kOPitch * 4 ? kLast : 8 * kOPitch * 4;
  // Items per SM.  A multiple of four: an SM's registers lie in four parts, and what
  // does not fit its part waits (64 decoding rows in e4m3: 84 us with 12, 112 with
  // 14 of the 144 registers that 14 would leave).
  static constexpr int kWarps = DP <= 64 ? (NT <= 2 ? 16 : 12) : NT == 1 || (E4 && NT == 2) ? 12 : 8;
};

// The 8 x 8 matrix of 16-bit numbers whose rows the lanes' quads hold, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// How a few rows of any lengths are cut into at most `budget` parts that run side
// by side, none much longer than another (the lanes of a warp together): item
// `idx` is part `split` of row `b`, of its `parts`.  A lane keeps rows 4 lane ..
// 4 lane + 3.  A row of w groups makes max(1, ceil(w / c)) parts, and c is the
// least, searched upwards from sum w / budget, for which the budget holds: it
// does for c = sum w / (budget - B) + 1, since sum ceil(w / c) <= sum w / c + B.
__device__ __forceinline__ void cut_groups(const PagedParams &P, int idx, int &b, int &split, int &parts) {
  const int lane = threadIdx.x % 32;
  uint32_t w[kKeep], sum = 0, top = 0;
#pragma unroll
  for (int q = 0; q < kKeep; ++q) {
    const int r = lane * kKeep + q;
    w[q] = 0;
    if (r < P.B) {
      int n;
      const int c = paged_queries(P, r, n);
      if (c > 0) w[q] = Keys(P, n, n + c).n;  // < 2^24, and the sum < 2^31 (kMaxCutTokens)
    }
    sum += w[q];
    top = max(top, w[q]);
  }
  sum = __reduce_add_sync(FULL_MASK, sum);
  top = __reduce_max_sync(FULL_MASK, top);
  const uint32_t least = max((top + P.splits - 1) / P.splits, static_cast<uint32_t>(P.min_groups));
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
  // the row of item idx: running sums over the lanes
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
  int row = lane * kKeep, cnt = 0;
#pragma unroll
  for (int q = 0; q < kKeep; ++q) {
    if (q < kKeep - 1 && row == lane * kKeep + q && k >= n[q]) {
      k -= n[q];
      ++row;
    } else if (row == lane * kKeep + q) {
      cnt = static_cast<int>(n[q]);
    }
  }
  const int src = __ffs(owner) - 1;
  b = __shfl_sync(FULL_MASK, row, src);
  split = __shfl_sync(FULL_MASK, static_cast<int>(k), src);
  parts = __shfl_sync(FULL_MASK, cnt, src);
}

// Items: x: KV head and block of kM query rows, y: part, z: row; or (cut by a
// budget) y: a part of any row, z: 0.
template <int CT, int DP, int NT>
__global__ void __launch_bounds__(32, PagedRowCfg<CT, DP, NT>::kWarps) paged_rows_kernel(const __grid_constant__ PagedParams P) {
  using C = PagedRowCfg<CT, DP, NT>;
  constexpr bool E4 = C::E4;
  constexpr bool BF = CT == SPEC_BF16;
  constexpr int kSteps = DP / 16;  // steps of the scores' contraction, tiles of the sums' rows
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *const qsm = smem + C::kQAt;
  float *const qfac = reinterpret_cast<float *>(qsm + C::kM * C::kQPitch);
  const int lane = threadIdx.x, quad = lane / 4, j4 = lane % 4;

  // --- the item: KV heads first (the heads of a token lie side by side in
  // memory, so the items that run together read whole entries), then parts
  if (static_cast<int>(blockIdx.y) < P.check) {  // (a launch less: 64 decoding rows 86 -> 84 us)
    const int r = P.budget > 0 ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x == 0 ? blockIdx.z : P.B;
    if (r >= P.B) return;
    int n;
    const int c = paged_queries(P, r, n);
    const bool fine = __all_sync(FULL_MASK, pages_there(P, r, n, c, lane, 32)) && c >= 0;
    if (lane == 0) {
      P.rowinfo[r] = fine ? c : kRowBadSlot;
      if (P.row_status) P.row_status[r] = fine ? 0 : SPEC_ROW_BAD_SLOT;
    }
    return;
  }
  const int item = blockIdx.y - P.check;
  int b = blockIdx.z, split = item, parts = P.splits;
  const int blk = blockIdx.x / static_cast<unsigned>(P.H), g = blockIdx.x - blk * P.H;
  const int blocks = gridDim.x / P.H;
  if (P.budget > 0) {
    cut_groups(P, split, b, split, parts);
    if (b < 0) {
      grid_dependency_wait();
      return;
    }
    if (split == 0 && g == 0 && lane == 0) P.parts_of[b] = make_int2(item, parts);  // (one block of query rows)
  }
  const int r0 = blk * C::kM, nrows = P.N * P.G;
  const bool cut = P.budget > 0;
  const long long flag = cut ? static_cast<long long>(item) * P.H + g : ((static_cast<long long>(b) * P.H + g) * blocks + blk) * P.splits + split;
  int n;
  const int cnt = paged_queries(P, b, n);
  const bool tree = P.anc != nullptr;
  if (tree) grid_dependency_wait();
  const int q_first = r0 / P.G, q_last = min((r0 + C::kM - 1) / P.G, P.N - 1);
  // Lane i knows query row i of the block (kM <= 32): its output row (-1 past
  // the last), whether it has a use, where its query is, and its position.
  int my_row = -1, my_pos = 0;
  bool my_use = false;
  long long my_q = 0;
  {
    const int r = r0 + lane;
    if (lane < C::kM && r < nrows) {
      const int t = r / P.G, h = g * P.G + (r - t * P.G);
      my_row = (b * P.N + t) * P.Hq + h;
      my_use = t < cnt;
      my_q = b * P.qs[0] + t * P.qs[1] + h * P.qs[2];
      my_pos = n + (tree && my_use && P.rowinfo[b] > 0 ? P.depth[static_cast<size_t>(b) * P.N + t] : tree ? 0 : t);
    }
  }
  const int end = cnt <= q_first ? 0 : tree ? n + cnt : n + min(cnt, q_last + 1);  // tokens below it
  const int p0 = tree ? n : n + q_first, p1 = tree ? n + cnt : n + q_last;          // positions lie in p0 .. p1
  const Keys keys(P, p0, end);
  int g0 = 0, g1 = keys.n;
  if (P.splits > 1) {
    const int per = max(P.min_groups, (keys.n + parts - 1) / parts);
    g0 = min(keys.n, split * per);
    g1 = min(keys.n, g0 + per);
  }
  if (g0 >= g1 && P.splits > 1) {  // nothing here
    if (lane == 0) P.oflag[flag] = 0;
    if (my_row >= 0) P.ml[cut ? flag * C::kM + lane : static_cast<long long>(split) * P.rows + my_row] = make_float2(-INFINITY, -INFINITY);
    grid_dependency_wait();
    return;
  }

  // --- the queries' loads, before the many of the ring
  constexpr int QL = DP / 8, kRows = 32 / QL, kPass = C::kM / kRows;  // lanes per row, rows per pass
  const int qc = lane % QL;
  uint4 u[kPass];
  {
    const bool vec = reinterpret_cast<uintptr_t>(P.q) % 16 == 0 && P.qs[0] % 8 == 0 && P.qs[1] % 8 == 0 && P.qs[2] % 8 == 0;
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int rr = i * kRows + lane / QL;
      const bool use = __shfl_sync(FULL_MASK, my_use, rr);
      const long long off = __shfl_sync(FULL_MASK, my_q, rr);
      u[i] = make_uint4(0, 0, 0, 0);
      if (use && qc * 8 < P.D) {
        const unsigned short *q = static_cast<const unsigned short *>(P.q) + off + qc * 8;
        if (vec) {
          u[i] = __ldg(reinterpret_cast<const uint4 *>(q));
        } else {
          u[i].x = q[0] | static_cast<uint32_t>(q[1]) << 16;
          u[i].y = q[2] | static_cast<uint32_t>(q[3]) << 16;
          u[i].z = q[4] | static_cast<uint32_t>(q[5]) << 16;
          u[i].w = q[6] | static_cast<uint32_t>(q[7]) << 16;
        }
      }
    }
  }

  // --- the ring of groups: lanes over a token's 16-byte pieces, then over tokens
  const uint32_t ring = smem_u32(smem);
  constexpr int L = DP * C::kEsz / 16, kPer = kGroup * L / 32, kStep = 32 / L;
  const int pc = lane % L, row0 = lane / L;
  const bool col = pc * 16 < P.D * C::kEsz;
  const int32_t *const trow = P.table + static_cast<size_t>(b) * P.columns;
  const long long piece = static_cast<long long>(g) * P.D * C::kEsz + (col ? pc * 16 : 0);
  // lane i: where group base + i of the part starts in its plane (-1: on no page)
  long long where = -1;
  auto look_up = [&](int base) {
    where = -1;
    if (base + lane < g1) {
      const int t = keys.token(base + lane), j = t / P.page, pg = __ldg(trow + j);
      if (pg >= 0 && pg < P.pages) where = pg * P.page_stride + (t - j * P.page) * P.tok_stride;
    }
  };
  if (P.D < DP) {  // the columns past the head vector stay zero: no copy writes them
    for (int i = lane; i < C::kStages * C::kStage / 16; i += 32) *reinterpret_cast<uint4 *>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  auto issue = [&](int gi, int st) {
    if (gi < g1) {
      if ((gi - g0) % 32 == 0) look_up(gi);
      const long long at = __shfl_sync(FULL_MASK, where, (gi - g0) % 32);
      const uint32_t base = ring + st * C::kStage + row0 * C::kPitch + pc * 16;
      const int left = at < 0 ? 0 : end - keys.token(gi);
      const long long off = at < 0 ? 0 : at + piece + row0 * P.tok_stride;
      if (col) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool on = row0 + i * kStep < left;
          const long long o = on ? off + i * kStep * P.tok_stride : 0;
          cp_async16_zfill(base + i * kStep * C::kPitch, P.k + o, on);
          cp_async16_zfill(base + C::kPlane + i * kStep * C::kPitch, P.v + o, on);
        }
      }
      if constexpr (E4) {  // scale words: lanes 0-15 the keys', 16-31 the values' of token lane % 16
        const bool on = lane % kGroup < left;
        const long long o = on ? at + lane % kGroup * P.tok_stride + static_cast<long long>(P.H) * P.D + (g & ~3) : 0;
        cp_async4_zfill(ring + st * C::kStage + 2 * C::kPlane + lane * 4, (lane < kGroup ? P.k : P.v) + o, on);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(g0 + s, s);

  // --- queries into the last ring slot; fp16 for an e4m3 cache: a row far
  // outside fp16's range is brought into it by a power of two
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int rr = i * kRows + lane / QL;
    float fac = 1.f;
    if (E4 && P.qbf16) {
      const float x[8] = {bf16_lo(u[i].x), bf16_hi(u[i].x), bf16_lo(u[i].y), bf16_hi(u[i].y),
                          bf16_lo(u[i].z), bf16_hi(u[i].z), bf16_lo(u[i].w), bf16_hi(u[i].w)};
      uint32_t a = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
      for (int o = QL / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL_MASK, a, o));
      float by = 1.f;
      const int e = static_cast<int>(a >> 23) - 127;
      if (a != 0 && a < 0x7f800000u && (e < -4 || e > 14)) {
        const int up = max(-126, min(126, -e));
        by = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
        fac = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      }
      u[i] = make_uint4(pack16<false>(x[0] * by, x[1] * by), pack16<false>(x[2] * by, x[3] * by),
                        pack16<false>(x[4] * by, x[5] * by), pack16<false>(x[6] * by, x[7] * by));
    }
    if (qc == 0) qfac[rr] = fac;
    *reinterpret_cast<uint4 *>(qsm + rr * C::kQPitch + qc * 16) = u[i];
  }
  __syncwarp();

  // Fragments.  The contraction over d may run in any order as long as Q and
  // K agree: for codes a thread takes DP/4 consecutive d (a few 16-byte
  // reads), for 16-bit entries the order ldmatrix gives.
  uint32_t qf[C::kHeld ? NT : 1][kSteps][2];
#pragma unroll
  for (int t = 0; t < (C::kHeld ? NT : 0); ++t)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d0 = E4 ? j4 * (DP / 4) + s * 4 : s * 16 + j4 * 2, d1 = E4 ? d0 + 2 : d0 + 8;
      qf[t][s][0] = *reinterpret_cast<const uint32_t *>(qsm + (t * 8 + quad) * C::kQPitch + d0 * 2);
      qf[t][s][1] = *reinterpret_cast<const uint32_t *>(qsm + (t * 8 + quad) * C::kQPitch + d1 * 2);
    }
  // the thread's query rows 8 t + 2 j4 and the next: factors, for the masks tokens and positions
  float rf[NT][2];
  int qtok[NT][2], qpos[NT][2];
  bool scaled = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rr = t * 8 + 2 * j4 + c;
      rf[t][c] = qfac[rr];
      scaled = scaled || rf[t][c] != 1.f;
      qtok[t][c] = min((r0 + rr) / P.G, P.N - 1);
      qpos[t][c] = __shfl_sync(FULL_MASK, my_pos, rr);
    }
  scaled = E4 && __any_sync(FULL_MASK, scaled);
  auto fragment = [&](int t, int s, uint32_t (&f)[2]) {
    if constexpr (C::kHeld) {
      f[0] = qf[t][s][0], f[1] = qf[t][s][1];
    } else {
      const uint32_t at = smem_u32(qsm) + (t * 8 + quad) * C::kQPitch + (E4 ? j4 * (DP / 4) + s * 4 : s * 16 + j4 * 2) * 2;
      if constexpr (E4) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(f[0]), "=r"(f[1]) : "r"(at) : "memory");
      } else {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(f[0]) : "r"(at) : "memory");
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(f[1]) : "r"(at + 16) : "memory");
      }
    }
  };
  if (C::kHeld && P.D < DP) {  // the slot's padding columns were queries
    __syncwarp();
    for (int i = lane; i < C::kStage / 16; i += 32) *reinterpret_cast<uint4 *>(qsm + i * 16) = make_uint4(0, 0, 0, 0);
  }
  __syncwarp();

  // sums: tile s of 16 columns d; components d of the quad and the other half's,
  // each of the thread's two query rows
  float o[kSteps][NT][4];
  // l counts in units of 2^mx, o in units of 2^mv (one and the same for 16-bit entries)
  float mx[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mx[t][0] = mx[t][1] = mv[t][0] = mv[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[s][t][c] = 0.f;
  }

  bool odd = false;
  int st = 0;
  for (int gi = g0; gi < g1; ++gi) {
    issue(gi + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t kst = ring + st * C::kStage, vst = kst + C::kPlane, sst = kst + 2 * C::kPlane;
    const int tb = keys.token(gi);
    // some query of the block does not see some token of the group
    const bool masked = tb + kGroup - 1 > (tree ? n - 1 : p0) || (tb + kGroup > P.sinks && tb < window_from(P, p1));
    // --- in masked groups, values that are not finite are taken out
    if (masked) {
      bool bad = false;
      for (int tk = 0; tk < kGroup; ++tk)
#pragma unroll
        for (int i = 0; i < (DP * C::kEsz + 127) / 128; ++i) {  // words of a head vector
          if ((i * 32 + lane) * 4 >= P.D * C::kEsz) continue;
          const uint32_t at = vst + tk * C::kPitch + (i * 32 + lane) * 4;
          uint32_t w;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
          uint32_t r = w;
          if constexpr (E4) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if ((w >> (8 * c) & 127u) == 127u) r &= ~(255u << (8 * c));
          } else {
            constexpr uint32_t top = BF ? 0x7f80u : 0x7c00u;
            if ((w & top) == top) r &= 0xffff0000u;
            if ((w >> 16 & top) == top) r &= 0x0000ffffu;
          }
          if (r != w) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(r) : "memory");
            bad = true;
          }
        }
      odd = __any_sync(FULL_MASK, bad) || odd;
      __syncwarp();
    }
    // lane i < 16: token i's key scale; lane 16 + i: its value scale
    uint32_t byte = 0;
    if constexpr (E4) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(sst + lane * 4) : "memory");
      byte = w >> (8 * (g & 3)) & 255u;
      // value vectors of NaN: the keys alone decide the softmax, and the NaN comes in with the values
      const unsigned nans = __ballot_sync(FULL_MASK, byte == 255u) >> kGroup;
      if (nans) {
        for (int tk = 0; tk < kGroup; ++tk) {
          if (!(nans >> tk & 1u)) continue;
          if (masked)  // not every query sees it: put into the answers of those that do
            odd = true;
          else if (lane * 4 < P.D)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(vst + tk * C::kPitch + lane * 4), "r"(0x7f7f7f7fu) : "memory");
        }
        __syncwarp();
      }
    }
    // --- scores: tokens quad (c < 2) and quad + 8, query rows 8 t + 2 j4 + c % 2
    // (two sums each, for shorter chains)
    float x[NT][4], x2[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[t][c] = x2[t][c] = 0.f;
    if constexpr (E4) {
      const uint32_t at = kst + quad * C::kPitch + j4 * (DP / 4);
#pragma unroll
      for (int s0 = 0; s0 < kSteps; s0 += 4) {
        uint32_t w[2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[hf][0]), "=r"(w[hf][1]), "=r"(w[hf][2]), "=r"(w[hf][3])
                       : "r"(at + hf * 8 * C::kPitch + s0 * 4)
                       : "memory");
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t kf[4] = {e4m3x2_to_f16x2(w[0][s]), e4m3x2_to_f16x2(w[1][s]), e4m3x2_to_f16x2_hi(w[0][s]), e4m3x2_to_f16x2_hi(w[1][s])};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t f[2];
            fragment(t, s0 + s, f);
            mma16816<false>(s & 1 ? x2[t] : x[t], kf, f[0], f[1]);
          }
        }
      }
    } else {
      // matrices: (tokens 0-7, d 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
      const uint32_t at = kst + (lane % 16) * C::kPitch + (lane / 16) * 16;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t kf[4];
        ldmatrix_x4(kf, at + s * 32);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t f[2];
          fragment(t, s, f);
          mma16816<BF>(s & 1 ? x2[t] : x[t], kf, f[0], f[1]);
        }
      }
    }
    // the values' loads, ahead of what their weights take
    constexpr int kCols = DP / 8;  // codes: columns of a quad
    constexpr bool kEarly = E4 ? NT == 1 : NT <= 3;
    uint32_t vw[E4 ? kCols / 8 : 1][4][2], vf[E4 ? 1 : kSteps][4];
    auto load_codes = [&](int n0) {
      // of tokens 2 j4, 2 j4 + 1, 8 + 2 j4, 9 + 2 j4 the quad's columns
#pragma unroll
      for (int t = 0; t < 4; ++t)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(vw[n0 / 8][t][0]), "=r"(vw[n0 / 8][t][1])
                     : "r"(vst + ((t / 2) * 8 + 2 * j4 + t % 2) * C::kPitch + quad * kCols + n0)
                     : "memory");
    };
    // matrices: (tokens 0-7, d 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15), each transposed
    const uint32_t vat = vst + ((lane / 16) * 8 + lane % 8) * C::kPitch + ((lane / 8) % 2) * 16;
    if constexpr (kEarly && E4) {
#pragma unroll
      for (int n0 = 0; n0 < kCols; n0 += 8) load_codes(n0);
    } else if constexpr (kEarly) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) ldmatrix_x4_trans(vf[s], vat + s * 32);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[t][c] += x2[t][c];
    // --- to base-2 exponents
    float ve[2] = {0.f, 0.f};  // the values' scale exponents of the thread's two tokens
    if constexpr (E4) {
      const float mine = lane < kGroup ? P.scale * e4m3_scale(byte) : byte == 255u ? 0.f : scale_exponent(byte);
      float ks[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        ks[hf] = __shfl_sync(FULL_MASK, mine, quad + 8 * hf);
        ve[hf] = __shfl_sync(FULL_MASK, mine, kGroup + quad + 8 * hf);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[t][c] *= ks[c >> 1];
      if (scaled) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[t][c] *= rf[t][c & 1];
      }
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[t][c] *= P.scale;
    }
    if (masked) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tk = tb + quad + 8 * (c >> 1);
          if (tk >= end || !paged_sees(P, b, qtok[t][c & 1], n, qpos[t][c & 1], tk)) x[t][c] = -INFINITY;
        }
    }
    // --- softmax.  A row's references follow its maxima only when these have
    // grown by more than 2^kPaLazy (weights up to that are as exact), whatever
    // other rows' do: nothing of a row depends on its neighbours in the block.
    bool grown = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float a = fmaxf(x[t][c], x[t][2 + c]);
        grown = grown || a > mx[t][c] + kPaLazy || mx[t][c] == -INFINITY;
        if constexpr (E4) grown = grown || fmaxf(x[t][c] + ve[0], x[t][2 + c] + ve[1]) > mv[t][c] + kPaLazy;
      }
    if (__any_sync(FULL_MASK, grown)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float al[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a = fmaxf(x[t][c], x[t][2 + c]);
#pragma unroll
          for (int q = 4; q < 32; q <<= 1) a = fmaxf(a, __shfl_xor_sync(FULL_MASK, a, q));
          al[c] = 1.f;
          if (a > mx[t][c] + kPaLazy || (mx[t][c] == -INFINITY && a > -INFINITY)) {
            al[c] = ex2(mx[t][c] - a);
            l[t][c] *= al[c];
            mx[t][c] = a;
          }
          if constexpr (E4) {
            a = fmaxf(x[t][c] + ve[0], x[t][2 + c] + ve[1]);
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) a = fmaxf(a, __shfl_xor_sync(FULL_MASK, a, q));
            al[c] = 1.f;
            if (a > mv[t][c] + kPaLazy || (mv[t][c] == -INFINITY && a > -INFINITY)) {
              al[c] = ex2(mv[t][c] - a);
              mv[t][c] = a;
            }
          }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[s][t][c] *= al[c & 1];
      }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float ref = mx[t][c] == -INFINITY ? 0.f : mx[t][c], rev = mv[t][c] == -INFINITY ? 0.f : mv[t][c];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float &y = x[t][2 * hf + c];
          const float w = ex2(y - ref);
          l[t][c] += w;
          y = E4 ? ex2(y + (ve[hf] - rev)) : w;
        }
      }
      pf[t][0] = transpose8(pack16<BF>(x[t][0], x[t][1]));
      pf[t][1] = transpose8(pack16<BF>(x[t][2], x[t][3]));
    }
    // --- values times weights
    if constexpr (E4) {
      // a tile takes two of the quad's columns
#pragma unroll
      for (int n0 = 0; n0 < kCols; n0 += 8) {
        if constexpr (!kEarly) load_codes(n0);
        const uint32_t(&w)[4][2] = vw[n0 / 8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          // bytes i, i + 1 of two tokens: (t0 i, t1 i, t0 i+1, t1 i+1)
          const uint32_t sel = i % 4 == 0 ? 0x5140u : 0x7362u;
          const uint32_t lo = __byte_perm(w[0][i / 4], w[1][i / 4], sel);
          const uint32_t hi = __byte_perm(w[2][i / 4], w[3][i / 4], sel);
          const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2_hi(lo), e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2_hi(hi)};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<false>(o[(n0 + i) / 2][t], a, pf[t][0], pf[t][1]);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if constexpr (!kEarly) ldmatrix_x4_trans(vf[s], vat + s * 32);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816<BF>(o[s][t], vf[s], pf[t][0], pf[t][1]);
      }
    }
    __syncwarp();
    st = st == C::kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait_all();
  allow_dependents();  // the join's blocks may take the places that come free
  grid_dependency_wait();  // the row's check
  const bool usable = P.check > 0 || P.rowinfo[b] >= 0;  // (else the join leaves the row out)
  odd = __any_sync(FULL_MASK, odd);
  if (P.splits > 1 && lane == 0) P.oflag[flag] = odd;
  // Eight query rows at a time through shared memory, so that a row is written
  // by the whole warp.
  float *const buf = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d = E4 ? quad * (DP / 8) + 2 * s + (c >> 1) : s * 16 + quad + 8 * (c >> 1);
        buf[(2 * j4 + (c & 1)) * C::kOPitch + d] = o[s][t][c];
      }
    // the rows' statistics: in the lanes of quad 0, as in all others
    float mr[2], zr[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float a = l[t][c];
#pragma unroll
      for (int q = 4; q < 32; q <<= 1) a += __shfl_xor_sync(FULL_MASK, a, q);
      mr[c] = E4 ? mv[t][c] : mx[t][c];
      zr[c] = a != 0.f ? mx[t][c] + log2f(a) : -INFINITY;
    }
    __syncwarp();
#pragma unroll 1
    for (int row = 0; row < 8; ++row) {
      const int rr = t * 8 + row;
      const int orow = __shfl_sync(FULL_MASK, my_row, rr), pos = __shfl_sync(FULL_MASK, my_pos, rr);
      const bool use = __shfl_sync(FULL_MASK, my_use, rr);
      const float m = __shfl_sync(FULL_MASK, row & 1 ? mr[1] : mr[0], row / 2);
      float z = __shfl_sync(FULL_MASK, row & 1 ? zr[1] : zr[0], row / 2);
      if (orow < 0) break;  // rows past the last
      const bool some = usable && use && z != -INFINITY;
      if (!some) z = -INFINITY;
      const float4 y = *reinterpret_cast<const float4 *>(buf + row * C::kOPitch + min(lane * 4, DP - 4));
      if (P.splits > 1) {
        const long long at = cut ? flag * C::kM + rr : static_cast<long long>(split) * P.rows + orow;
        if (lane == 0) P.ml[at] = some ? make_float2(m, z) : make_float2(-INFINITY, -INFINITY);
        if (some && lane * 4 < P.D) *reinterpret_cast<float4 *>(P.part + at * P.D + lane * 4) = y;
        continue;
      }
      if (lane == 0 && P.lse) P.lse[orow] = kLn2 * z;
      if (lane * 4 >= P.D) continue;
      const float w = some ? ex2(m - z) : 0.f;
      float a[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = some ? a[e] * w : 0.f;
        if (some && odd) a[e] += paged_odd_sum<CT>(P, b, min((r0 + rr) / P.G, P.N - 1), cnt, n, pos, g, lane * 4 + e);
      }
      *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(P.out) + static_cast<long long>(orow) * P.D + lane * 4) =
          P.qbf16 ? make_uint2(pack16<true>(a[0], a[1]), pack16<true>(a[2], a[3])) : make_uint2(pack16<false>(a[0], a[1]), pack16<false>(a[2], a[3]));
    }
  }
}

// ------------------------------------------------------------------- join
// One warp per output row: the weights of the parts, then their sum, eight parts'
// loads at a time.
template <int CT, bool BF>
__global__ void __launch_bounds__(kPaJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams P) {
  const int lane = threadIdx.x % 32;
  const long long r = static_cast<long long>(blockIdx.x) * (kPaJoinThreads / 32) + threadIdx.x / 32;
  grid_dependency_wait();
  if (r >= P.rows) return;
  const int b = static_cast<int>(r / (static_cast<long long>(P.N) * P.Hq));
  const int qt = static_cast<int>(r / P.Hq) - b * P.N, h = static_cast<int>(r % P.Hq);
  const int c = P.rowinfo[b];
  const bool on = qt < c;
  float Z = -INFINITY;
  bool gone = false;  // a part's kernel gave up waiting: the row is flagged and its answer left empty
  float2 ml = make_float2(-INFINITY, -INFINITY);  // this lane's part (there are 32 at most)
  const int g = h / P.G, row = qt * P.G + h % P.G;  // the row among its KV head's
  int parts = P.splits;
  long long at0 = r, step = P.rows, flag0, fstep = 1;  // the first part, and from one to the next; so with the flags
  if (P.budget > 0) {
    const int2 of = P.parts_of[b];
    parts = of.y;
    flag0 = static_cast<long long>(of.x) * P.H + g;
    fstep = P.H;
    at0 = flag0 * P.oblk + row;
    step = static_cast<long long>(P.H) * P.oblk;
  } else {
    flag0 = ((static_cast<long long>(b) * P.H + g) * ((P.N * P.G + P.oblk - 1) / P.oblk) + row / P.oblk) * P.splits;
  }
  if (on && lane < parts) ml = P.ml[at0 + lane * step];
  gone = __any_sync(FULL_MASK, __float_as_uint(ml.y) == kTimeoutBits);
  if (gone && lane == 0 && P.row_status) P.row_status[b] = SPEC_ROW_TIMEOUT;
  Z = ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) Z = fmax_nan(Z, __shfl_xor_sync(FULL_MASK, Z, o));
  const float zref = Z == -INFINITY ? 0.f : Z;
  const float S = gone ? 0.f : warp_sum(ex2(ml.y - zref));
  const float z = S == 0.f ? -INFINITY : zref + log2f(S);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};  // columns 4 lane .. 4 lane + 3
  if (S != 0.f) {
    const float wl = ex2(ml.x - z);
    unsigned todo = __ballot_sync(FULL_MASK, ml.y != -INFINITY);
    while (todo) {
      float4 x[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = todo ? __ffs(todo) - 1 : -1;
        todo &= todo - 1;
        w[j] = __shfl_sync(FULL_MASK, wl, k & 31);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < 0)
          w[j] = 0.f;
        else if (lane * 4 < P.D)
          x[j] = *reinterpret_cast<const float4 *>(P.part + (at0 + k * step) * P.D + lane * 4);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[0] = fmaf(w[j], x[j].x, acc[0]);
        acc[1] = fmaf(w[j], x[j].y, acc[1]);
        acc[2] = fmaf(w[j], x[j].z, acc[2]);
        acc[3] = fmaf(w[j], x[j].w, acc[3]);
      }
    }
    if (__any_sync(FULL_MASK, lane < parts && P.oflag[flag0 + lane * fstep])) {
      const int n = P.kv_len[b], p = n + (P.anc ? P.depth[static_cast<size_t>(b) * P.N + qt] : qt);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane * 4 + i < P.D) acc[i] += paged_odd_sum<CT>(P, b, qt, c, n, p, g, lane * 4 + i);
    }
  }
  if (lane * 4 < P.D)
    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(P.out) + r * P.D + lane * 4) =
        make_uint2(pack16<BF>(acc[0], acc[1]), pack16<BF>(acc[2], acc[3]));
  if (lane == 0 && P.lse) P.lse[r] = kLn2 * z;
}

// -------------------------------------------------------------------- host
template <int CT, int DP, int NT>
cudaError_t launch_rows(const PagedParams &p, cudaStream_t s) {
  using C = PagedRowCfg<CT, DP, NT>;
  const int blocks = (p.N * p.G + C::kM - 1) / C::kM;
  const dim3 grid(p.H * blocks, (p.budget > 0 ? p.budget : p.splits) + p.check, p.budget > 0 ? 1 : p.B);
  const cudaError_t e = allow_smem<paged_rows_kernel<CT, DP, NT>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(paged_rows_kernel<CT, DP, NT>, grid, 32, C::kSmem, s, p.check == 0, p);
}

template <int CT, int DP>
cudaError_t launch_rows_n(const PagedParams &p, cudaStream_t s) {
  if (p.oblk == 8) return launch_rows<CT, DP, 1>(p, s);
  if (p.oblk == 16) return launch_rows<CT, DP, 2>(p, s);
  if (p.oblk == 24) return launch_rows<CT, DP, 3>(p, s);
  return launch_rows<CT, DP, 4>(p, s);
}

template <int CT>
cudaError_t launch_rows_d(const PagedParams &p, cudaStream_t s) {
  return p.D <= 64 ? launch_rows_n<CT, 64>(p, s) : launch_rows_n<CT, 128>(p, s);
}

// Items of the rows kernel that run on an SM at a time.
int rows_per_sm(int ct, int D, int oblk) {
  auto of = [&](auto c) {
    constexpr int CT = decltype(c)::value;
    if (D <= 64) return oblk <= 16 ? PagedRowCfg<CT, 64, 1>::kWarps : PagedRowCfg<CT, 64, 4>::kWarps;
    return oblk == 8 ? PagedRowCfg<CT, 128, 1>::kWarps : oblk == 16 ? PagedRowCfg<CT, 128, 2>::kWarps : PagedRowCfg<CT, 128, 4>::kWarps;
  };
  return ct == SPEC_E4M3 ? of(std::integral_constant<int, SPEC_E4M3>()) : of(std::integral_constant<int, SPEC_BF16>());
}

struct PagedPlan {
  bool tile;           // paged_tile_kernel
  int splits, budget, oblk, W;
  size_t rows, info_at, count_at, anc_at, depth_at, flag_at, ml_at, part_at, bytes;
};

size_t pa_round(size_t x) { return (x + 255) / 256 * 256; }
bool pa_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes and types (no pointers).
spec_status check_paged(const spec_paged_attention_args *a) {
  const long long most = 0x7fffffffLL;
  if (a->q_dtype != SPEC_BF16 && a->q_dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  if (a->cache_dtype != SPEC_E4M3 && a->cache_dtype != a->q_dtype) return SPEC_ERR_DTYPE;
  const size_t entry = spec_kv_entry_bytes(a->heads, a->head_dim, a->cache_dtype);
  if (entry == 0 || a->B < 0 || a->B > 65535 || a->N < 0 || a->q_heads < 1 || a->q_heads % a->heads) return SPEC_ERR_SHAPE;
  if (a->columns < 1 || a->page_size < 16 || a->page_size > SPEC_MAX_PAGE || a->page_size % 16 || a->num_pages < 0) return SPEC_ERR_SHAPE;
  // positions leave room for a window's end and a group past the last token
  if (static_cast<long long>(a->columns) * a->page_size > most - 4096 || static_cast<long long>(a->num_pages) * a->page_size > most)
    return SPEC_ERR_SHAPE;
  if (a->parent && a->N > SPEC_MAX_TREE_NODES) return SPEC_ERR_SHAPE;
  if (a->N > 0 && static_cast<long long>(a->B) * a->N >= most / 256 / a->q_heads) return SPEC_ERR_SHAPE;
  if (static_cast<long long>(a->N) * (a->q_heads / a->heads) > most / 2) return SPEC_ERR_SHAPE;
  if (a->page_stride < (a->num_pages > 1 ? 16 : 0) || a->page_stride >= 1LL << 40 || a->tok_stride < static_cast<int64_t>(entry) || a->tok_stride >= 1LL << 27) return SPEC_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (a->q_stride[i] < 0) return SPEC_ERR_SHAPE;
  if (!std::isfinite(a->scale * kLog2e) || a->window < 0 || a->sinks < 0) return SPEC_ERR_ARG;
  return SPEC_OK;
}

PagedPlan plan_paged(const spec_paged_attention_args *a) {
  PagedPlan p = {};
  const long long G = a->q_heads / a->heads, rows1 = a->N * G;
  p.rows = static_cast<size_t>(a->B) * a->N * a->q_heads;
  // More than 32 query rows per KV head would read the keys again for each 32.  (fp16
  // queries over codes go that way all the same: as bf16, which the tile kernel
  // turns codes into, they would lose three bits.)
  p.tile = rows1 > 32 && !(a->cache_dtype == SPEC_E4M3 && a->q_dtype == SPEC_F16);
  p.oblk = p.tile ? 256 : static_cast<int>(std::min<long long>(32, (rows1 + 7) / 8 * 8));
  const long long blocks = (rows1 + p.oblk - 1) / p.oblk, items = a->B * a->heads * blocks;
  // tokens that an item may see
  long long tokens = static_cast<long long>(a->columns) * a->page_size;
  if (a->window > 0) tokens = std::min(tokens, static_cast<long long>(a->window) + a->sinks + p.oblk / G + 1 + 2 * kGroup);
  if (p.tile) {
    // one CTA per SM runs through items: the fewest rounds of items times their
    // blocks of 128 keys, an item's ends counting as two
    const long long n = (tokens + 127) / 128;
    long long best = -1;
    p.splits = 1;
    for (long long s = 1; s <= std::min<long long>(n, 32); ++s) {
      const long long cost = (items * s + kPagedSms - 1) / kPagedSms * ((n + s - 1) / s + 2) + (s > 1 ? 3 : 0);
      if (best < 0 || cost < best) best = cost, p.splits = static_cast<int>(s);
    }
  } else {
    const long long want = (8LL * kPagedSms * 2 + items - 1) / items;
    p.splits = static_cast<int>(std::max<long long>(1, std::min<long long>({want, (tokens + kGroup - 1) / kGroup, 32})));
    // A few rows are cut by a budget of parts, all items side by side.
    const long long budget = static_cast<long long>(rows_per_sm(a->cache_dtype, a->head_dim, p.oblk)) * kPagedSms / a->heads;
    if (blocks == 1 && a->B <= kMaxCutRows && budget > a->B && tokens <= kMaxCutTokens) {
      p.budget = static_cast<int>(budget);
      p.splits = static_cast<int>(std::min<long long>({32, (tokens + kGroup - 1) / kGroup, budget - a->B + 1}));
    }
  }
  p.W = a->parent ? (a->N + 31) / 32 : 0;
  const size_t q = static_cast<size_t>(a->B) * a->N;
  size_t at = 0;
  p.info_at = at;
  at += pa_round(static_cast<size_t>(a->B) * 4);
  p.count_at = at;
  at += pa_round(static_cast<size_t>(a->B) * 8);
  p.anc_at = at;
  at += pa_round(q * p.W * 4);
  p.depth_at = at;
  at += pa_round(a->parent ? q * 4 : 0);
  // parts times what each has: rows of answers, or (by a budget) of a block
  size_t flags = static_cast<size_t>(items) * p.splits, part_rows = p.splits * p.rows;
  if (p.budget > 0) {
    flags = static_cast<size_t>(std::min<long long>(p.budget, static_cast<long long>(a->B) * p.splits)) * a->heads;
    part_rows = flags * p.oblk;
  }
  p.flag_at = at;
  if (p.splits > 1) at += pa_round(flags * 4);
  p.ml_at = at;
  if (p.splits > 1) at += pa_round(part_rows * sizeof(float2));
  p.part_at = at;
  if (p.splits > 1) at += pa_round(part_rows * a->head_dim * 4);
  p.bytes = at + 256;
  return p;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_paged_attention_workspace_size(const spec_paged_attention_args *a) {
  if (!a || check_paged(a) != SPEC_OK) return 0;
  if (a->B == 0 || a->N == 0) return 256;
  return plan_paged(a).bytes;
}

spec_status spec_paged_attention(const spec_paged_attention_args *a, void *out, float *lse, int32_t *row_status,
                                 void *ws, size_t ws_bytes, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const spec_status st = check_paged(a);
  if (st != SPEC_OK) return st;
  if (!pa_aligned(a->k, 16) || !pa_aligned(a->v, 16) || a->page_stride % 16 || a->tok_stride % 16 || !pa_aligned(a->q, 2) ||
      !pa_aligned(out, 16) || !pa_aligned(lse, 16) || !pa_aligned(row_status, 4) || !pa_aligned(a->block_table, 4) ||
      !pa_aligned(a->kv_len, 4) || !pa_aligned(a->count, 4) || !pa_aligned(a->parent, 4))
    return SPEC_ERR_ALIGN;
  if (a->B == 0 || a->N == 0) return SPEC_OK;
  if (!a->q || !out || !a->kv_len || !a->block_table || ((!a->k || !a->v) && a->num_pages > 0)) return SPEC_ERR_NULL;
  const PagedPlan plan = plan_paged(a);
  if (!ws || !pa_aligned(ws, 256) || ws_bytes < plan.bytes) return SPEC_ERR_WORKSPACE;
  char *w = static_cast<char *>(ws);
  PagedParams p = {};
  p.k = static_cast<const unsigned char *>(a->k);
  p.v = static_cast<const unsigned char *>(a->v);
  if (a->num_pages == 0) p.k = p.v = reinterpret_cast<const unsigned char *>(w);  // nothing of it is read
  p.page_stride = a->page_stride;
  p.tok_stride = a->tok_stride;
  p.page = a->page_size;
  p.pages = a->num_pages;
  p.columns = a->columns;
  p.table = a->block_table;
  p.q = a->q;
  for (int i = 0; i < 3; ++i) p.qs[i] = a->q_stride[i];
  p.scale = a->scale * kLog2e;
  p.B = a->B;
  p.N = a->N;
  p.Hq = a->q_heads;
  p.H = a->heads;
  p.G = a->q_heads / a->heads;
  p.D = a->head_dim;
  p.kv_len = a->kv_len;
  p.count = a->count;
  p.window = a->window > 0 ? a->window : 0x7fffffff;
  p.sinks = a->window > 0 ? a->sinks : 0;
  p.W = plan.W;
  p.rows = static_cast<int>(plan.rows);
  p.splits = plan.splits;
  p.budget = plan.splits > 1 ? plan.budget : 0;
  p.parts_of = reinterpret_cast<int2 *>(w + plan.count_at);
  p.min_groups = 1;  // (one token under a window of 128: 14.0 us with four, 11.7 so)
  p.oblk = plan.oblk;
  p.ml = reinterpret_cast<float2 *>(w + plan.ml_at);
  p.part = reinterpret_cast<float *>(w + plan.part_at);
  p.oflag = reinterpret_cast<int32_t *>(w + plan.flag_at);
  p.out = out;
  p.lse = lse;
  p.row_status = row_status;
  p.qbf16 = a->q_dtype == SPEC_BF16;
  p.wait_limit_ns = spec_get_wait_timeout_ns();
  p.force_timeout = force_wait_timeout();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t *info = reinterpret_cast<int32_t *>(w + plan.info_at);
  uint32_t *anc = reinterpret_cast<uint32_t *>(w + plan.anc_at);
  int32_t *depth = reinterpret_cast<int32_t *>(w + plan.depth_at);
  p.rowinfo = info;
  if (!plan.tile && !a->parent && p.splits > 1) {
    const int across = p.H * ((p.N * p.G + p.oblk - 1) / p.oblk);  // blocks of a blockIdx.y
    p.check = p.budget > 0 ? (p.B + across - 1) / across : 1;
  } else {
    paged_check_kernel<<<p.B, kCheckThreads, 0, s>>>(p, a->parent, anc, depth);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  }
  if (a->parent) p.anc = anc, p.depth = depth;
  const int ct = a->cache_dtype;
  cudaError_t e = plan.tile         ? launch_paged_tile(p, ct, s)
                  : ct == SPEC_E4M3 ? launch_rows_d<SPEC_E4M3>(p, s)
                  : ct == SPEC_BF16 ? launch_rows_d<SPEC_BF16>(p, s)
                                    : launch_rows_d<SPEC_F16>(p, s);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  if (p.splits == 1) return SPEC_OK;
  const dim3 grid((p.rows + kPaJoinThreads / 32 - 1) / (kPaJoinThreads / 32));
  auto join = [&](auto kernel) { return launch_after(kernel, grid, kPaJoinThreads, 0, s, true, p); };
  e = ct == SPEC_BF16  ? join(paged_join_kernel<SPEC_BF16, true>)
      : ct == SPEC_F16 ? join(paged_join_kernel<SPEC_F16, false>)
      : p.qbf16        ? join(paged_join_kernel<SPEC_E4M3, true>)
                       : join(paged_join_kernel<SPEC_E4M3, false>);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
