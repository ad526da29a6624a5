// prefix_attention.cu -- the verify pass's attention over a shared prefix and
// each row's own cache (spec_prefix_attention): the entry point, the tree
// mask, the kernel for few query rows and the join of the parts.
//
//  attn_mask_kernel -- draft trees only: checks each row's parents and turns
//    them into ancestor bits, one thread per node walking to the root.
//  attn_tile_kernel (prefix_attention_tile.cu) -- many query rows.
//  attn_rows_kernel -- 16 or 32 query rows (the query heads of one KV head and
//    the tokens of one row; for the prefix, of all rows) against a range of
//    tokens, one warp.  Bound by the cache's bytes, so what matters is bytes in
//    flight: every warp streams its range through a ring of asynchronous
//    copies of its own.  e4m3 codes are turned into fp16 in registers on the
//    way to the tensor cores (exact), scales go into the scores and the
//    weights.  With this few rows the synchronous matrix instructions keep up
//    with memory; tensor memory's tiles of 128 rows would be mostly padding.
//  attn_join_kernel -- one warp per query row adds up the parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "internal.h"

namespace sv {
namespace {

constexpr int kSms = 152;           // parts are sized for this many SMs
constexpr float kRowLazy = 8.f;
constexpr float kExponentGrowth = 20.f, kFarApart = -INFINITY;
constexpr int kMaskThreads = 256;
constexpr int kJoinThreads = 128;

// ---------------------------------------------------------------- tree mask
// Latency alone: three dependent loads and a walk up the deepest path, under the
// conversion and tile kernels' own starts.  Where the tile kernel writes the
// answers itself, row_status is written here, so that no CTA's "fine" can come
// after another's timeout (chains: parent is NULL, and that is all there is to do).
__global__ void __launch_bounds__(kMaskThreads) attn_mask_kernel(const int32_t *parent, const int32_t *kv_len,
                                                                 const int32_t *count, long long slots, int N, int W,
                                                                 uint32_t *anc, int32_t *rowinfo, int32_t *row_status) {
  __shared__ int par[SPEC_MAX_TREE_NODES];
  const int b = blockIdx.x, tid = threadIdx.x;
  allow_dependents();
  const int n = kv_len[b], c = count ? count[b] : N;
  const bool slot_ok = n >= 0 && c >= 0 && c <= N && static_cast<long long>(n) + c <= slots;
  const int used = parent ? max(0, min(c, N)) : 0;
  bool ok = true;
  for (int i = tid; i < used; i += kMaskThreads) {
    const int p = parent[static_cast<size_t>(b) * N + i];
    par[i] = p;
    ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
  }
  ok = __syncthreads_and(ok);
  if (tid == 0) rowinfo[b] = !ok ? kRowBadParent : !slot_ok ? kRowBadSlot : c;
  if (tid == 0 && row_status) row_status[b] = !ok ? SPEC_ROW_BAD_PARENT : !slot_ok ? SPEC_ROW_BAD_SLOT : 0;
  if (!ok || !slot_ok) return;
  for (int i = tid; i < used; i += kMaskThreads) {
    uint32_t *row = anc + (static_cast<size_t>(b) * N + i) * W;
    int w = W - 1, j = i;
    uint32_t bits = 0;
    while (j >= 0) {  // indexes fall strictly on the way up
      while (w > (j >> 5)) {
        row[w--] = bits;
        bits = 0;
      }
      bits |= 1u << (j & 31);
      j = par[j];
    }
    row[w] = bits;  // w == 0: the root is in word 0
  }
}

// ------------------------------------------------------------- row kernel
template <int CT, int DP, int MT>
struct RowCfg {
  static constexpr bool E4 = CT == SPEC_E4M3;
  static constexpr int kEsz = E4 ? 1 : 2;
  static constexpr int kM = 16 * MT;                        // query rows
  static constexpr int kBlk = 16;                           // tokens per block
  static constexpr int kStages = 3;
  static constexpr int kPitch = DP * kEsz + 16;             // bytes of one token in a ring slot
  static constexpr int kPlane = kBlk * kPitch;              // K or V of a block
  static constexpr int kScales = E4 ? 2 * kBlk * 4 : 0;     // scale words, K then V
  static constexpr int kTable = E4 ? kBlk * 16 : 0;         // what they come to, per token
  static constexpr int kStage = 2 * kPlane + kScales;
  static constexpr int kQPitch = DP * 2 + 16;
  static constexpr int kQ = kM * kQPitch + kM * 4;          // queries and factors, in the last slot before it is used
  static constexpr int kSmem = (kStages - 1) * kStage + (kStage > kQ ? kStage : kQ) + kTable;
  static constexpr int kWarps = MT == 2 || !E4 ? 8 : 12;    // items per SM: registers, and shared memory for 16-bit rings
};

// Registers bound it where head vectors are longer than 64: e4m3 items of 16 rows
// spill 252 bytes a thread, of 32 rows 536, 16-bit items of 32 rows 48.
// One warp per item and nothing shared between warps: 8 to 12 items run on an
// SM side by side, and while one starts or ends the others keep the memory
// busy.  (Four warps on one item and a join in shared memory: 52 us where this
// takes 35, 64 chains of 6 tokens over 33 K entries of 8 heads in bf16: 3.9 TB/s
// on the whole, 6.6 within the loop; all items start and end together.)
// Items: x: KV head and block of kM query rows, y: part, z: row (or, cut by a
// budget, y: a part of any row, z: 0), or one past the last for the prefix (whose
// query rows are those of all rows).
template <int CT, int DP, int MT>
__global__ void __launch_bounds__(32, RowCfg<CT, DP, MT>::kWarps) attn_rows_kernel(const __grid_constant__ AttnParams P, int own,
                                                                                   int pblocks, int oblocks) {
  using C = RowCfg<CT, DP, MT>;
  constexpr bool E4 = C::E4;
  constexpr bool BF = CT == SPEC_BF16;
  constexpr int kBlk = C::kBlk;
  constexpr int kSteps = DP / 16, kNt = DP / 8;  // k-steps of the scores, column tiles of the sums
  constexpr int kTt = kBlk / 8, kTs = kBlk / 16; // token tiles of the scores, k-steps of the sums
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *const qsm = smem + (C::kStages - 1) * C::kStage;
  float *const qfac = reinterpret_cast<float *>(qsm + C::kM * C::kQPitch);
  const int lane = threadIdx.x, quad = lane / 4, j4 = lane % 4;

  // --- the item: KV heads first (the heads of a token lie side by side in
  // memory, so the items that run together read whole entries), then parts
  int b = blockIdx.z, split = blockIdx.y;
  const int blk = blockIdx.x / static_cast<unsigned>(P.H), g = blockIdx.x - blk * P.H;
  const bool pre = b >= own;  // the prefix's items come after those of the `own` rows
  int t0 = 0, t1 = 0, len0 = 0, cnt = 0;   // tokens; own slots below len0 are seen by every query
  if (!pre && P.budget > 0) {
    int parts;
    cut_rows(P, split, b, split, parts, t0, t1);
    if (b >= 0 && split == 0 && blk == 0 && g == 0 && lane == 0) P.nparts[b] = parts;
  }
  if (b < 0 || blk >= (pre ? pblocks : oblocks) || split >= (pre ? P.psplits : P.osplits)) {  // the grid is a box
    grid_dependency_wait();
    return;
  }
  const int r0 = blk * C::kM;              // first query row of the block
  const int nrows = (pre ? P.B : 1) * P.N * P.G;
  const int slot = pre ? split : P.psplits + split;
  const long long flag = ((static_cast<long long>(b) * P.H + g) * oblocks + blk) * P.osplits + split;
  const unsigned char *kb, *vb;
  long long ts;
  if (pre) {
    t0 = split * P.pchunk;
    t1 = min(P.P, t0 + P.pchunk);
    kb = P.pk, vb = P.pv, ts = P.ptok_stride;
  } else {
    cnt = row_queries(P, b);
    len0 = __ldg(P.kv_len + b);
    if (cnt <= 0)
      t0 = t1 = 0;
    else if (P.budget > 0)
      t1 = min(t1, len0 + cnt);
    else
      own_range(P, len0 + cnt, split, t0, t1);
    kb = P.k + b * P.row_stride, vb = P.v + b * P.row_stride, ts = P.tok_stride;
    if (split == 0 && blk == 0 && g == 0 && lane == 0 && P.row_status)
      P.row_status[b] = cnt >= 0 ? 0 : cnt == kRowBadParent ? SPEC_ROW_BAD_PARENT : SPEC_ROW_BAD_SLOT;
  }
  // Lane i knows query row i of the block (kM <= 32): its output row (-1 past
  // the last), its token, where its query is, whether it has a use.
  int my_row = -1;
  bool my_use = false;
  long long my_q = 0;
  {
    const int r = r0 + lane;
    if (lane < C::kM && r < nrows) {
      const int t = r / P.G, h = g * P.G + (r - t * P.G);
      const int qb = pre ? t / P.N : b, qt = pre ? t - qb * P.N : t;
      my_row = (qb * P.N + qt) * P.Hq + h;
      my_use = qt < (pre ? row_queries(P, qb) : cnt);
      my_q = qb * P.qs[0] + qt * P.qs[1] + h * P.qs[2];
    }
  }
  if (t0 >= t1) {  // nothing here (an empty part, or a row that cannot be used)
    if (!pre && lane == 0) P.oflag[flag] = 0;
    if (my_row >= 0) P.ml[static_cast<long long>(slot) * P.rows + my_row] = make_float2(-INFINITY, -INFINITY);
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

  // --- the ring of token blocks: lanes over a token's 16-byte pieces, then
  // over tokens; pointers advance
  const uint32_t ring = smem_u32(smem);
  const int nblk = (t1 - t0 + kBlk - 1) / kBlk;
  constexpr int L = DP * C::kEsz / 16, kPer = kBlk * L / 32, kStep = 32 / L;
  const int pc = lane % L, row0 = lane / L;
  const bool col = pc * 16 < P.D * C::kEsz;
  const long long first = static_cast<long long>(t0 + row0) * ts + static_cast<long long>(g) * P.D * C::kEsz + (col ? pc * 16 : 0);
  const unsigned char *kp = kb + first, *vp = vb + first;
  const uint32_t step = static_cast<uint32_t>(ts) * kStep;  // fits: strides are below 2^27
  const long long jump = ts * kBlk;
  // scale words: lanes 0-15 the keys', 16-31 the values' of token lane % 16
  const unsigned char *sp = nullptr;
  if constexpr (E4)
    sp = (lane < kBlk ? kb : vb) + static_cast<long long>(t0 + lane % kBlk) * ts + static_cast<long long>(P.H) * P.D + (g & ~3);
  if (P.D < DP) {  // the columns past the head vector stay zero: no copy writes them
    for (int i = lane; i < C::kStages * C::kStage / 16; i += 32) *reinterpret_cast<uint4 *>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  auto issue = [&](int blkno, int st) {
    if (blkno < nblk) {
      const uint32_t base = ring + st * C::kStage + row0 * C::kPitch + pc * 16;
      const int left = t1 - (t0 + blkno * kBlk);
      if (left >= kBlk) {
        if (col) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            cp_async16_zfill(base + i * kStep * C::kPitch, kp + static_cast<uint64_t>(step) * i, true);
            cp_async16_zfill(base + C::kPlane + i * kStep * C::kPitch, vp + static_cast<uint64_t>(step) * i, true);
          }
        }
      } else if (col) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool on = row0 + i * kStep < left;
          cp_async16_zfill(base + i * kStep * C::kPitch, on ? kp + static_cast<uint64_t>(step) * i : kb, on);
          cp_async16_zfill(base + C::kPlane + i * kStep * C::kPitch, on ? vp + static_cast<uint64_t>(step) * i : vb, on);
        }
      }
      kp += jump;
      vp += jump;
      if constexpr (E4) {
        const bool on = lane % kBlk < left;
        cp_async4_zfill(ring + st * C::kStage + 2 * C::kPlane + lane * 4, on ? sp : kb, on);
        sp += jump;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s, s);

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
  uint32_t qf[MT][kSteps][4];
  float rf[MT][2];
  bool scaled = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int rr = mt * 16 + hf * 8 + quad;
      rf[mt][hf] = qfac[rr];
      scaled = scaled || rf[mt][hf] != 1.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d0 = E4 ? j4 * (DP / 4) + s * 4 : s * 16 + j4 * 2;
        const int d1 = E4 ? d0 + 2 : d0 + 8;
        qf[mt][s][hf] = *reinterpret_cast<const uint32_t *>(qsm + rr * C::kQPitch + d0 * 2);
        qf[mt][s][2 + hf] = *reinterpret_cast<const uint32_t *>(qsm + rr * C::kQPitch + d1 * 2);
      }
    }
  }
  scaled = __any_sync(FULL_MASK, scaled);
  if (P.D < DP) {  // the slot's padding columns were queries
    __syncwarp();
    for (int i = lane; i < C::kStage / 16; i += 32) *reinterpret_cast<uint4 *>(qsm + i * 16) = make_uint4(0, 0, 0, 0);
  }
  __syncwarp();
  // each thread's rows, for the mask of the pass's own tokens
  int qtok[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) qtok[mt][hf] = min((r0 + mt * 16 + hf * 8 + quad) / P.G, P.N - 1);

  float o[MT][kNt][4];
  float mx[MT][2], l[MT][2];
  float E = kMinExponent;  // l counts in units of 2^(mx - E), E the largest scale exponent so far
  // what E may grow to after the first block that holds more than the least
  // scales; kFarApart: scales lie too far apart for such units
  float limit = INFINITY;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    mx[mt][0] = mx[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[mt][n][c] = 0.f;
  }

  bool odd = false;
  int st = 0;
  for (int blkno = 0; blkno < nblk; ++blkno) {
    issue(blkno + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t kst = ring + st * C::kStage, vst = kst + C::kPlane, sst = kst + 2 * C::kPlane;
    const int tb = t0 + blkno * kBlk;
    // --- scores: token n * 8 + 2 j4 + {0, 1} of rows quad and quad + 8
    float x[MT][kTt][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < kTt; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[mt][n][c] = 0.f;
    if constexpr (E4) {
#pragma unroll
      for (int n = 0; n < kTt; ++n) {
        const uint32_t at = kst + (n * 8 + quad) * C::kPitch + j4 * (DP / 4);
#pragma unroll
        for (int s0 = 0; s0 < kSteps; s0 += 4) {
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(at + s0 * 4)
                       : "memory");
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t b0 = e4m3x2_to_f16x2(w[s]), b1 = e4m3x2_to_f16x2_hi(w[s]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816<false>(x[mt][n], qf[mt][s0 + s], b0, b1);
          }
        }
      }
    } else {
      // matrices: (tokens 0-7, d 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
      const uint32_t at = kst + ((lane / 16) * 8 + lane % 8) * C::kPitch + ((lane / 8) % 2) * 16;
#pragma unroll
      for (int n = 0; n < kTt; n += 2)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t kf[4];
          ldmatrix_x4(kf, at + n * 8 * C::kPitch + s * 32);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<BF>(x[mt][n], qf[mt][s], kf[0], kf[1]);
            mma16816<BF>(x[mt][n + 1], qf[mt][s], kf[2], kf[3]);
          }
        }
    }
    // --- to base-2 exponents of the weights
    float ve[kTt][2], inv[kTt][2], rest[kTt][2];
    bool small = false;
    float dE = 0.f;
    if constexpr (E4) {
      // lane i < 16: token i's key scale; lane 16 + i: its value scale
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(sst + lane * 4) : "memory");
      const uint32_t byte = w >> (8 * (g & 3)) & 255u;
      const float e = scale_exponent(byte);
      const int most = __reduce_max_sync(FULL_MASK, lane < kBlk || byte == 255u ? -127 : static_cast<int>(byte) - 127);
      const float En = fmaxf(E, static_cast<float>(most));
      if (En > limit) limit = kFarApart;
      if (limit == INFINITY && most + 127 > static_cast<int>(kLeastScale)) limit = En + kExponentGrowth;
      dE = En - E;
      E = En;
      const bool none = byte == 255u, low = lane >= kBlk && e < E - kExponentSpan;
      if (__any_sync(FULL_MASK, low || none)) {
        small = __any_sync(FULL_MASK, low);
        if (__any_sync(FULL_MASK, low && byte > kLeastScale)) limit = kFarApart;
        // value vectors of NaN: the keys alone decide the softmax, and the NaN comes in with the values
        const unsigned nans = __ballot_sync(FULL_MASK, none) >> kBlk;
        for (int tk = 0; tk < kBlk; ++tk) {
          if (!(nans >> tk & 1u)) continue;
          if (!pre && tb + tk >= len0)  // one of the pass's own: put into the answers that see it
            odd = true;
          else if (lane * 4 < P.D)  // every query sees it
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(vst + tk * C::kPitch + lane * 4), "r"(0x7f7f7f7fu) : "memory");
        }
        __syncwarp();
      }
      const float ec = low ? E - kExponentSpan : none ? E : e;
      const uint32_t tab = smem_u32(smem) + C::kSmem - C::kTable;
      if (lane < kBlk)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(tab + lane * 16), "f"(P.scale * e4m3_scale(byte)) : "memory");
      else
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(tab + (lane - kBlk) * 16 + 8), "f"(ec), "f"(low ? ex2(e - ec) : 1.f) : "memory");
      __syncwarp();
      float ks[kTt][2];
#pragma unroll
      for (int n = 0; n < kTt; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float unused;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(ks[n][c]), "=f"(unused), "=f"(ve[n][c]), "=f"(rest[n][c])
                       : "r"(tab + (n * 8 + 2 * j4 + c) * 16)
                       : "memory");
          inv[n][c] = ex2(E - ve[n][c]);
        }
      if (scaled) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < kTt; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[mt][n][c] *= rf[mt][c >> 1];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < kTt; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[mt][n][c] = fmaf(x[mt][n][c], ks[n][c & 1], ve[n][c & 1]);
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < kTt; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[mt][n][c] *= P.scale;
    }
    // --- masks: the range's end, and the pass's own tokens
    const bool masked = tb + kBlk > t1 || (!pre && tb + kBlk > len0);
    if (masked) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < kTt; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int t = tb + n * 8 + 2 * j4 + (c & 1);
            bool see = t < t1;
            const int jn = t - len0;
            if (see && !pre && jn >= 0) {
              const int qi = qtok[mt][c >> 1];
              see = P.anc ? (__ldg(P.anc + (static_cast<size_t>(b) * P.N + qi) * P.W + (jn >> 5)) >> (jn & 31)) & 1 : jn <= qi;
            }
            if (!see) x[mt][n][c] = -INFINITY;
          }
    }
    // --- softmax.  A row's reference follows its maximum only when that has
    // grown by more than 2^kRowLazy (weights up to that are as exact).
    float tm[MT][2], al[MT][2], old[MT][2];
    bool grown = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float t = fmaxf(x[mt][0][2 * hf], x[mt][0][2 * hf + 1]);
#pragma unroll
        for (int n = 1; n < kTt; ++n) t = fmaxf(t, fmaxf(x[mt][n][2 * hf], x[mt][n][2 * hf + 1]));
        tm[mt][hf] = t;
        old[mt][hf] = mx[mt][hf];
        al[mt][hf] = 1.f;
        grown = grown || t > mx[mt][hf] + kRowLazy || mx[mt][hf] == -INFINITY;
      }
    const bool moved = __any_sync(FULL_MASK, grown);
    if (moved) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float t = tm[mt][hf];
          t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 1));
          t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 2));
          if (t > mx[mt][hf]) {
            al[mt][hf] = ex2(mx[mt][hf] - t);
            mx[mt][hf] = t;
          }
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          o[mt][n][0] *= al[mt][0];
          o[mt][n][1] *= al[mt][0];
          o[mt][n][2] *= al[mt][1];
          o[mt][n][3] *= al[mt][1];
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float ref = mx[mt][hf] == -INFINITY ? 0.f : mx[mt][hf];
        float add = 0.f;
#pragma unroll
        for (int n = 0; n < kTt; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float &y = x[mt][n][2 * hf + c];
            y = ex2(y - ref);
            // 0 * NaN: a token that is not seen adds nothing, whatever its scale
            if constexpr (E4)
              add += y == 0.f ? 0.f : y * inv[n][c];
            else
              add += y;
          }
        // old = -inf: nothing was summed yet
        const float ll = E4 && dE != 0.f ? (old[mt][hf] == -INFINITY ? 0.f : ex2(old[mt][hf] - ref + dE)) : al[mt][hf];
        l[mt][hf] = fmaf(l[mt][hf], ll, add);
      }
    if constexpr (E4) {
      if (small) {  // the rest of the factor of scales that far below the largest
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < kTt; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[mt][n][c] *= rest[n][c & 1];
      }
    }
    uint32_t pf[MT][kTs][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < kTs; ++s) {
        pf[mt][s][0] = pack16<BF>(x[mt][2 * s][0], x[mt][2 * s][1]);
        pf[mt][s][1] = pack16<BF>(x[mt][2 * s][2], x[mt][2 * s][3]);
        pf[mt][s][2] = pack16<BF>(x[mt][2 * s + 1][0], x[mt][2 * s + 1][1]);
        pf[mt][s][3] = pack16<BF>(x[mt][2 * s + 1][2], x[mt][2 * s + 1][3]);
      }
    // --- values of the pass's own tokens that are not finite: a query that
    // does not see them would get 0 * NaN.  They are taken out here and put
    // into the answers of the queries that see them when the parts are joined.
    if (masked && !pre) {
      bool bad = false;
      for (int tk = max(0, len0 - tb); tk < min(kBlk, t1 - tb); ++tk)
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
    // --- weights times values
    if constexpr (E4) {
      // tokens 2 j4, 2 j4 + 1, 8 + 2 j4, 9 + 2 j4 of columns quad * kNt + n
#pragma unroll
      for (int s = 0; s < kTs; ++s)
#pragma unroll
        for (int n0 = 0; n0 < kNt; n0 += 8) {
          uint32_t w[4][2];
#pragma unroll
          for (int t = 0; t < 4; ++t)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(w[t][0]), "=r"(w[t][1])
                         : "r"(vst + (s * 16 + (t / 2) * 8 + 2 * j4 + t % 2) * C::kPitch + quad * kNt + n0)
                         : "memory");
#pragma unroll
          for (int n = 0; n < 8; n += 2) {
            // bytes n, n + 1 of two tokens: (t0 n, t1 n, t0 n+1, t1 n+1)
            const uint32_t sel = n % 4 == 0 ? 0x5140u : 0x7362u;
            const uint32_t lo = __byte_perm(w[0][n / 4], w[1][n / 4], sel);
            const uint32_t hi = __byte_perm(w[2][n / 4], w[3][n / 4], sel);
            const uint32_t b0 = e4m3x2_to_f16x2(lo), b1 = e4m3x2_to_f16x2(hi);
            const uint32_t c0 = e4m3x2_to_f16x2_hi(lo), c1 = e4m3x2_to_f16x2_hi(hi);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<false>(o[mt][n0 + n], pf[mt][s], b0, b1);
              mma16816<false>(o[mt][n0 + n + 1], pf[mt][s], c0, c1);
            }
          }
        }
    } else {
      // matrices: (tokens 0-7, d 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
      const uint32_t at = vst + (lane % 16) * C::kPitch + (lane / 16) * 16;
#pragma unroll
      for (int s = 0; s < kTs; ++s)
#pragma unroll
        for (int n = 0; n < kNt; n += 2) {
          uint32_t vf[4];
          ldmatrix_x4_trans(vf, at + s * 16 * C::kPitch + n * 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<BF>(o[mt][n], pf[mt][s], vf[0], vf[1]);
            mma16816<BF>(o[mt][n + 1], pf[mt][s], vf[2], vf[3]);
          }
        }
    }
    __syncwarp();
    st = st == C::kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait_all();
  allow_dependents();  // the join's blocks may take the places that come free

  if (!pre && lane == 0) P.oflag[flag] = odd;
  if (E4 && limit == kFarApart) {
    if (my_row >= 0) {
      const int h = my_row % P.Hq, t = my_row / P.Hq, qb = t / P.N, qt = t - qb * P.N;
      const uint32_t *const anc = pre || !P.anc ? nullptr : P.anc + static_cast<size_t>(t) * P.W;
      exact_part(P, b, g, pre ? t0 : 0, pre ? t1 : 0, pre ? 0 : t0, pre ? 0 : t1, len0, cnt, qt, anc, my_use,
                 qb * P.qs[0] + qt * P.qs[1] + h * P.qs[2], my_row, slot, false);
    }
    grid_dependency_wait();
    return;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int rr = mt * 16 + hf * 8 + quad;
      const int orow = __shfl_sync(FULL_MASK, my_row, rr);
      const bool use = __shfl_sync(FULL_MASK, my_use, rr);
      float t = l[mt][hf];
      t += __shfl_xor_sync(FULL_MASK, t, 1);
      t += __shfl_xor_sync(FULL_MASK, t, 2);
      if (orow < 0) continue;
      const bool some = use && t != 0.f;
      const long long at = static_cast<long long>(slot) * P.rows + orow;
      if (j4 == 0)
        P.ml[at] = some ? make_float2(mx[mt][hf], mx[mt][hf] + log2f(t) - (E4 ? E : 0.f)) : make_float2(-INFINITY, -INFINITY);
      if (!some) continue;
      float *const to = P.part + at * P.D;
      if constexpr (E4) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int n = 0; n < kNt; n += 8) {
            if ((2 * j4 + c) * kNt + n >= P.D) continue;
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(o[mt][n + e][2 * hf + c]);
            st_global_v8(to + (2 * j4 + c) * kNt + n, y);
          }
      } else {
#pragma unroll
        for (int n = 0; n < kNt; ++n)
          if (n * 8 < P.D) *reinterpret_cast<float2 *>(to + n * 8 + 2 * j4) = make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
      }
    }
  // Started while the prefix's kernel ends, with which this one shares nothing:
  // it must not be over before that one, since the join waits for this one.
  grid_dependency_wait();
}

// ------------------------------------------------------------------- join
// One warp per output row: the weights of the parts, then their sum, eight parts'
// loads at a time (four: one microsecond more).  Bound by the parts' bytes, from
// L2 mostly, and by its start: 64 chains of 6 tokens (12288 rows) 10 us.
template <int CT, bool BF>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams P) {
  const int lane = threadIdx.x % 32;
  const long long r = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + threadIdx.x / 32;
  int nslots = P.psplits + P.osplits;
  const int b = static_cast<int>(r / (static_cast<long long>(P.N) * P.Hq));
  int n = 0;
  if (r < P.rows && !P.rowinfo) n = row_queries(P, b);  // inputs: no need to wait for the kernels before
  grid_dependency_wait();
  if (r >= P.rows) return;
  if (P.rowinfo) n = row_queries(P, b);
  if (P.budget > 0) nslots = P.psplits + P.nparts[b];
  const int qt = static_cast<int>(r / P.Hq) - b * P.N, h = static_cast<int>(r % P.Hq);
  const bool on = qt < n;
  float Z = -INFINITY;
  bool gone = false;  // a part's kernel gave up: the row is flagged and its answer left empty
  float2 ml0 = make_float2(-INFINITY, -INFINITY);  // this lane's first part
  if (on)
    for (int s = lane; s < nslots; s += 32) {
      const float2 x = P.ml[static_cast<long long>(s) * P.rows + r];
      if (s < 32) ml0 = x;
      const float z = x.y;
      gone = gone || __float_as_uint(z) == kTimeoutBits;
      Z = fmaxf(Z, z);
    }
  gone = __any_sync(FULL_MASK, gone);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) Z = fmaxf(Z, __shfl_xor_sync(FULL_MASK, Z, o));
  const float zref = Z == -INFINITY ? 0.f : Z;
  float S = 0.f;
  if (gone && lane == 0 && P.row_status) P.row_status[b] = SPEC_ROW_TIMEOUT;
  if (on && !gone) {
    S = ex2(ml0.y - zref);
    for (int s = lane + 32; s < nslots; s += 32) S += ex2(P.ml[static_cast<long long>(s) * P.rows + r].y - zref);
  }
  S = warp_sum(S);
  const float z = S == 0.f ? -INFINITY : zref + log2f(S);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};  // columns 4 lane .. 4 lane + 3
  if (S != 0.f)
    for (int s0 = 0; s0 < nslots; s0 += 32) {
      float2 ml = ml0;
      if (s0 > 0) ml = s0 + lane < nslots ? P.ml[static_cast<long long>(s0 + lane) * P.rows + r] : make_float2(-INFINITY, -INFINITY);
      const float wl = ex2(ml.x - z);
      // the parts that left a sum, eight at a time: their loads overlap
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
            x[j] = *reinterpret_cast<const float4 *>(P.part + (static_cast<long long>(s0 + k) * P.rows + r) * P.D + lane * 4);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[0] = fmaf(w[j], x[j].x, acc[0]);
          acc[1] = fmaf(w[j], x[j].y, acc[1]);
          acc[2] = fmaf(w[j], x[j].z, acc[2]);
          acc[3] = fmaf(w[j], x[j].w, acc[3]);
        }
      }
    }
  // values that are not finite, of the pass's tokens that this query sees
  if (S != 0.f) {
    const int g = h / P.G, blocks = (P.N * P.G + P.oblk - 1) / P.oblk;
    const int32_t *flag = P.oflag + ((static_cast<long long>(b) * P.H + g) * blocks + (qt * P.G + h % P.G) / P.oblk) * P.osplits;
    bool odd = false;
    for (int s = lane; s < nslots - P.psplits; s += 32) odd = odd || flag[s];
    if (__any_sync(FULL_MASK, odd)) {
      const int len0 = P.kv_len[b];
      for (int j = 0; j < n; ++j) {
        const bool see = P.anc ? P.anc[(static_cast<size_t>(b) * P.N + qt) * P.W + (j >> 5)] >> (j & 31) & 1u : j <= qt;
        if (!see) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane * 4 + i < P.D) acc[i] += odd_value<CT>(P, b, len0 + j, g, lane * 4 + i);
      }
    }
  }
  if (lane * 4 < P.D)
    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(P.out) + r * P.D + lane * 4) =
        make_uint2(pack16<BF>(acc[0], acc[1]), pack16<BF>(acc[2], acc[3]));
  if (lane == 0 && P.lse) P.lse[r] = kLn2 * z;
}

// -------------------------------------------------------------------- host
template <int CT, int DP, int MT>
cudaError_t launch_rows(const AttnParams &p, bool prefix, cudaStream_t s) {
  using C = RowCfg<CT, DP, MT>;
  const int pblocks = static_cast<int>((static_cast<long long>(p.B) * p.N * p.G + C::kM - 1) / C::kM);
  const int oblocks = (p.N * p.G + C::kM - 1) / C::kM;
  const int blocks = std::max(oblocks, prefix ? pblocks : 0);
  const int zown = p.budget > 0 ? 1 : p.B;
  const dim3 grid(p.H * blocks, std::max(p.budget > 0 ? p.budget : p.osplits, prefix ? p.psplits : 1), zown + (prefix ? 1 : 0));
  const cudaError_t e = allow_smem<attn_rows_kernel<CT, DP, MT>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(attn_rows_kernel<CT, DP, MT>, grid, 32, C::kSmem, s, p.next, p, zown, pblocks, oblocks);
}

// Items of the rows kernel that run on an SM at a time.
int rows_per_sm(int dtype, int oblk) {
  if (dtype == SPEC_E4M3) return oblk == 16 ? RowCfg<SPEC_E4M3, 128, 1>::kWarps : RowCfg<SPEC_E4M3, 128, 2>::kWarps;
  return oblk == 16 ? RowCfg<SPEC_BF16, 128, 1>::kWarps : RowCfg<SPEC_BF16, 128, 2>::kWarps;
}

// 16 query rows an item where no item would use more (half the sums and
// registers), else 32.
bool two_row_tiles(int B, int N, int G, bool prefix) { return N * G > 16 || (prefix && static_cast<long long>(B) * N * G > 16); }

template <int CT>
cudaError_t launch_rows_d(const AttnParams &p, bool prefix, cudaStream_t s) {
  const bool two = two_row_tiles(p.B, p.N, p.G, prefix);
  if (p.D <= 64) return two ? launch_rows<CT, 64, 2>(p, prefix, s) : launch_rows<CT, 64, 1>(p, prefix, s);
  return two ? launch_rows<CT, 128, 2>(p, prefix, s) : launch_rows<CT, 128, 1>(p, prefix, s);
}

struct AttnPlan {
  int psplits, pchunk, osplits, min_chunk, budget, W;
  bool ptile, otile;  // attn_tile_kernel for the prefix, for the own entries
  bool fuse, direct;  // own items take the prefix too; and nothing is left to join
  bool widen;         // an e4m3 prefix is turned into fp16 first
  int oblk;           // query rows per own item
  size_t rows, anc_at, info_at, flag_at, count_at, ml_at, part_at, wide_at, scale_at, far_at, bytes;
};

size_t at_round(size_t x) { return (x + 255) / 256 * 256; }
bool at_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes and types (no pointers).
spec_status check_attention(const spec_attention_args *a) {
  const spec_kv_cache &c = a->cache;
  if (a->q_dtype != SPEC_BF16 && a->q_dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  if (c.dtype != SPEC_E4M3 && c.dtype != a->q_dtype) return SPEC_ERR_DTYPE;
  spec_status st = check_kv_cache(c);
  if (st != SPEC_OK) return st;
  if (a->prefix_len < 0 || a->prefix_len > 0x7fffffffLL - 4096) return SPEC_ERR_SHAPE;
  if (a->prefix_len > 0) {
    if (a->prefix.dtype != c.dtype) return SPEC_ERR_DTYPE;
    st = check_kv_cache(a->prefix);
    if (st != SPEC_OK) return st;
    if (a->prefix.heads != c.heads || a->prefix.head_dim != c.head_dim || a->prefix.rows < 1 ||
        a->prefix.slots < a->prefix_len)
      return SPEC_ERR_SHAPE;
  }
  if (a->N < 0 || a->N > SPEC_MAX_TREE_NODES || a->q_heads < 1 || a->q_heads % c.heads) return SPEC_ERR_SHAPE;
  if (static_cast<long long>(c.rows) * a->N >= 0x7fffffffLL / 256 / a->q_heads) return SPEC_ERR_SHAPE;
  if (c.slots > 0x7fffffffLL - 4096) return SPEC_ERR_SHAPE;
  // the kernels step over a few tokens at a time in 32 bits
  if (c.tok_stride >= 1LL << 27 || (a->prefix_len > 0 && a->prefix.tok_stride >= 1LL << 27)) return SPEC_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (a->q_stride[i] < 0) return SPEC_ERR_SHAPE;
  if (!std::isfinite(a->scale)) return SPEC_ERR_ARG;
  return SPEC_OK;
}

// Which kernel, and how the keys are cut into parts.
AttnPlan plan_attention(const spec_attention_args *a) {
  AttnPlan p = {};
  const spec_kv_cache &c = a->cache;
  const long long G = a->q_heads / c.heads;
  const long long q = static_cast<long long>(c.rows) * a->N;
  p.rows = static_cast<size_t>(q) * a->q_heads;
  // more than 32 query rows per KV head would read the keys again for each 32
  p.ptile = q * G > 32;
  p.otile = a->N * G > 32;
  // rows kernel: 8 items per SM, no part under 64 tokens
  auto row_parts = [](long long blocks, long long tokens) {
    const long long want = (8 * kSms + blocks - 1) / blocks;
    return static_cast<int>(std::max<long long>(1, std::min<long long>({want, (tokens + 63) / 64, 64})));
  };
  // tile kernel (one item per SM at a time): the fewest rounds of items times
  // their blocks of 128 tokens, an item's start and end counting as three
  auto tile_parts = [](long long blocks, long long tokens) {
    const long long n = (tokens + 127) / 128;
    long long best = -1;
    int parts = 1;
    for (long long s = 1; s <= std::min<long long>(n, 64); ++s) {
      const long long cost = (blocks * s + kSms - 1) / kSms * ((n + s - 1) / s + 3);
      if (best < 0 || cost < best) best = cost, parts = static_cast<int>(s);
    }
    return parts;
  };
  // A tree's queries that nearly fill the row tiles take the prefix in the same
  // item as the row's own entries: queries are read once and, uncut, nothing
  // has to be joined.  Rows packed across the batch would save the padding only.
  const long long rows1 = a->N * G, padded = (rows1 + 127) / 128 * 128;
  p.fuse = p.otile && a->prefix_len > 0 && 4 * rows1 >= 3 * padded;
  if (a->prefix_len > 0 && !p.fuse) {
    p.psplits = p.ptile ? tile_parts(c.heads * ((q * G + 255) / 256), a->prefix_len)
                        : row_parts(c.heads * ((q * G + 31) / 32), a->prefix_len);
    const int unit = p.ptile ? 128 : 64;
    p.pchunk = static_cast<int>(((a->prefix_len + p.psplits - 1) / p.psplits + unit - 1) / unit * unit);
    p.psplits = static_cast<int>((a->prefix_len + p.pchunk - 1) / p.pchunk);
  }
  p.oblk = p.otile ? 256 : two_row_tiles(c.rows, a->N, static_cast<int>(G), a->prefix_len > 0 && !p.ptile) ? 32 : 16;
  const long long oblocks = (a->N * G + p.oblk - 1) / p.oblk;
  const long long oitems = c.rows * c.heads * oblocks;
  p.osplits = p.otile ? tile_parts(oitems, c.slots + (p.fuse ? a->prefix_len : 0)) : row_parts(oitems, c.slots);
  p.min_chunk = p.otile ? 128 : 64;
  if (!p.otile && oitems >= 2 * kSms) {
    // Rows differ in length.  A few rows are cut by a budget of parts so that
    // all items run side by side; more than kMaxCutRows are not cut.  That is well
    // where rows are alike (200 rows of 500 e4m3 entries, 8 heads of 128: 56 us, 0.55
    // of their bytes' time), not where one is long: 30000 entries in one of 200 rows
    // take 2.7 ms, in one of 128, where they make four parts, 0.77.
    const long long budget = rows_per_sm(c.dtype, p.oblk) * kSms / (c.heads * oblocks);
    p.osplits = 1;
    if (c.rows <= kMaxCutRows && budget > c.rows && c.slots < 1LL << 28) {
      p.budget = static_cast<int>(budget);
      p.osplits = static_cast<int>(std::min<long long>({std::max<long long>(1, (c.slots + 63) / 64), budget / c.rows * 4, 64}));
    }
  }
  p.direct = p.otile && p.osplits == 1 && p.psplits == 0;
  p.W = (a->N + 31) / 32;
  size_t at = 0;
  p.anc_at = at;
  at += at_round(static_cast<size_t>(q) * p.W * 4);
  p.info_at = at;
  at += at_round(static_cast<size_t>(c.rows) * 4);
  p.flag_at = at;
  at += at_round(static_cast<size_t>(c.rows) * c.heads * oblocks * p.osplits * 4);
  p.count_at = at;
  at += at_round(static_cast<size_t>(c.rows) * 4);
  p.ml_at = at;
  const size_t slots = static_cast<size_t>(p.psplits) + p.osplits;
  at += at_round(slots * p.rows * sizeof(float2));
  p.part_at = at;
  at += at_round(slots * p.rows * c.head_dim * 4);
  // An e4m3 prefix that several blocks of 256 query rows read is converted once
  // (two blocks: 4 us for the conversion of 8192 tokens of 8 heads where it saves 8)
  const long long readers = p.fuse ? c.rows * oblocks : p.ptile ? (q * G + 255) / 256 : 0;
  p.widen = c.dtype == SPEC_E4M3 && a->prefix_len > 0 && readers >= 2;
  if (p.widen) {
    p.wide_at = at;
    at += at_round(static_cast<size_t>(a->prefix_len) * c.heads * c.head_dim * 4);
    p.scale_at = at;
    at += at_round(static_cast<size_t>((a->prefix_len + 127) / 128) * c.heads * 2 * 4);
    p.far_at = at;
    at += at_round(static_cast<size_t>((a->prefix_len + 127) / 128) * c.heads * 2 * 4);
  }
  p.bytes = at + 256;
  return p;
}

}  // namespace

cudaError_t launch_attn_rows(const AttnParams &p, int ctype, bool prefix, cudaStream_t s) {
  if (ctype == SPEC_E4M3) return launch_rows_d<SPEC_E4M3>(p, prefix, s);
  if (ctype == SPEC_BF16) return launch_rows_d<SPEC_BF16>(p, prefix, s);
  return launch_rows_d<SPEC_F16>(p, prefix, s);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_prefix_attention_workspace_size(const spec_attention_args *a) {
  if (!a) return 0;
  spec_attention_args t = *a;  // sizes and types only
  t.cache.k = t.cache.v = t.prefix.k = t.prefix.v = nullptr;
  if (check_attention(&t) != SPEC_OK) return 0;
  if (a->cache.rows == 0 || a->N == 0) return 256;
  return plan_attention(a).bytes;
}

spec_status spec_prefix_attention(const spec_attention_args *a, void *out, float *lse, int32_t *row_status,
                                  void *ws, size_t ws_bytes, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const spec_status st = check_attention(a);
  if (st != SPEC_OK) return st;
  const spec_kv_cache &c = a->cache;
  if (!at_aligned(a->q, 2) || !at_aligned(out, 16) || !at_aligned(lse, 16) || !at_aligned(row_status, 4) ||
      !at_aligned(a->kv_len, 4) || !at_aligned(a->count, 4) || !at_aligned(a->parent, 4))
    return SPEC_ERR_ALIGN;
  if (c.rows == 0 || a->N == 0) return SPEC_OK;
  if (!a->q || !out || !a->kv_len || ((!c.k || !c.v) && c.slots > 0) ||
      (a->prefix_len > 0 && (!a->prefix.k || !a->prefix.v)))
    return SPEC_ERR_NULL;
  const AttnPlan plan = plan_attention(a);
  if (!ws || !at_aligned(ws, 256) || ws_bytes < plan.bytes) return SPEC_ERR_WORKSPACE;
  char *w = static_cast<char *>(ws);
  AttnParams p = {};
  p.k = static_cast<const unsigned char *>(c.k);
  p.v = static_cast<const unsigned char *>(c.v);
  p.row_stride = c.row_stride;
  p.tok_stride = c.tok_stride;
  p.slots = c.slots;
  p.P = static_cast<int>(a->prefix_len);
  if (p.P) {
    p.pk = static_cast<const unsigned char *>(a->prefix.k);
    p.pv = static_cast<const unsigned char *>(a->prefix.v);
    p.ptok_stride = a->prefix.tok_stride;
  }
  p.q = a->q;
  for (int i = 0; i < 3; ++i) p.qs[i] = a->q_stride[i];
  p.scale = a->scale * 1.442695040888963407f;
  p.B = c.rows;
  p.N = a->N;
  p.Hq = a->q_heads;
  p.H = c.heads;
  p.G = a->q_heads / c.heads;
  p.D = c.head_dim;
  p.kv_len = a->kv_len;
  p.count = a->count;
  p.W = plan.W;
  p.ml = reinterpret_cast<float2 *>(w + plan.ml_at);
  p.part = reinterpret_cast<float *>(w + plan.part_at);
  p.rows = static_cast<int>(plan.rows);
  p.psplits = plan.psplits;
  p.pchunk = plan.pchunk;
  p.osplits = plan.osplits;
  p.chunk = plan.otile ? 128 : 64;
  p.min_chunk = plan.min_chunk;
  p.budget = plan.budget;
  p.nparts = reinterpret_cast<int32_t *>(w + plan.count_at);
  p.oblk = plan.oblk;
  p.fuse = plan.fuse;
  p.oflag = reinterpret_cast<int32_t *>(w + plan.flag_at);
  p.out = out;
  p.lse = lse;
  p.row_status = row_status;
  p.qbf16 = a->q_dtype == SPEC_BF16;
  p.wait_limit_ns = spec_get_wait_timeout_ns();
  p.force_timeout = force_wait_timeout();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t *const status_here = plan.direct ? row_status : nullptr;
  if (a->parent || status_here) {
    uint32_t *anc = reinterpret_cast<uint32_t *>(w + plan.anc_at);
    int32_t *info = reinterpret_cast<int32_t *>(w + plan.info_at);
    attn_mask_kernel<<<p.B, a->parent ? kMaskThreads : 32, 0, s>>>(a->parent, a->kv_len, a->count, c.slots, p.N, p.W, anc, info,
                                                                   status_here);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
    if (a->parent) p.anc = anc;
    p.rowinfo = info;
  }
  if (plan.widen) {
    p.wide = reinterpret_cast<unsigned char *>(w + plan.wide_at);
    p.wide_scale = reinterpret_cast<float *>(w + plan.scale_at);
    p.wide_far = reinterpret_cast<int32_t *>(w + plan.far_at);
    if (launch_attn_widen(p, s) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  const bool prefix = p.P > 0;
  // The rows kernel may start while the tile kernel ends where both divide an
  // SM's memory alike, as with 16-bit rings (64 chains, bf16: 107 -> 103 us);
  // for codes each SM would have to be emptied in between (64 decoding rows: 79
  // -> 88 us), so there the kernels run one after the other.
  p.next = prefix && plan.ptile && !plan.otile && c.dtype != SPEC_E4M3;
  p.first = 1;
  if (prefix && plan.ptile && !plan.fuse) {
    if (launch_attn_tile(p, c.dtype, true, s) != cudaSuccess) return SPEC_ERR_CUDA;
    p.first = 0;
  }
  if (plan.otile) {
    p.direct = plan.direct;
    if (launch_attn_tile(p, c.dtype, false, s) != cudaSuccess) return SPEC_ERR_CUDA;
    if (plan.direct) return SPEC_OK;
    p.direct = 0;
  }
  if (!plan.otile &&
      launch_attn_rows(p, c.dtype, prefix && !plan.ptile, s) != cudaSuccess)
    return SPEC_ERR_CUDA;
  const dim3 grid((p.rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  auto join = [&](auto kernel) { return launch_after(kernel, grid, kJoinThreads, 0, s, true, p); };
  const cudaError_t e = c.dtype == SPEC_BF16  ? join(attn_join_kernel<SPEC_BF16, true>)
                        : c.dtype == SPEC_F16 ? join(attn_join_kernel<SPEC_F16, false>)
                        : p.qbf16             ? join(attn_join_kernel<SPEC_E4M3, true>)
                                              : join(attn_join_kernel<SPEC_E4M3, false>);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
