// paged_attention_tile.cu -- spec_paged_attention for many query rows: two tiles
// of 128 query rows (tokens and query heads of one KV head) against blocks of
// 128 keys, on the 5th-generation tensor cores.
//
// As in prefix_attention_tile.cu a CTA keeps two row tiles A and B, and the tensor
// cores work on one tile while a warpgroup does the other's softmax: scores,
// weights and sums stay in tensor memory (scores of A and B at columns 0 and 128,
// which the weights then take the place of; sums at 256 and 384), a thread owns
// a row, and sums are rescaled only when a row's maximum has grown by more than
// 2^8.  What differs:
//   - a block is eight groups of 16 keys, each from a page of its own, a box of the
//     cache as [page][token][head][number] (a group on no page lies past the last
//     one and comes as zeros); one warp looks the pages up, 32 at a time and ahead
//     of use, and asks for the boxes.  (With copies by 128 threads, 16 bytes at a
//     time, a prompt of 2 x 4096 tokens under a window of 1024 took 171 us, so 147;
//     134 with what follows);
//   - e4m3 codes are brought into a place of their own, and the producers make bf16
//     numbers of them, scale and all.  That is exact (4 bits of significand, and
//     bf16 has fp32's exponents), so scales may lie any distance apart;
//   - a CTA runs through many items (a prompt has hundreds of them), and the
//     roles do not meet between them.  One warp works the items out and hands
//     them on; the producers bring the next queries as soon as there is room, the
//     softmax sets the next item up while the last product is made, and the tensor
//     cores start on it while the answers are written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "paged_attention.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace {

constexpr int kBlk = 128;               // keys per block
constexpr int kBlkGroups = kBlk / kGroup;
// Warpgroups: the softmax of tiles A and B, producers, and one for the rest.  Codes
// have two of producers, for keys and for values, at the price of registers of the
// softmax: a prompt of 2 x 4096 tokens 230 us with one, 201 with two; in bf16, which
// has little for them to do, 145 us with one and 157 with two.
template <bool E4>
struct Team {
  static constexpr int kThreads = E4 ? 640 : 512;
  static constexpr int kProducers = E4 ? 2 : 1;
  static constexpr int kRest = 2 + kProducers;            // warpgroup of the rest:
  static constexpr int kIssueWarp = kRest * 4;            // (two, for tile A and tile B)
  static constexpr int kItemWarp = kRest * 4 + 2, kLoadWarp = kRest * 4 + 3;
  static constexpr int kLaunchRegs = E4 ? 96 : 128;       // 65536 / kThreads
  static constexpr int kSoftmaxRegs = E4 ? 144 : 184, kOtherRegs = E4 ? 64 : 72;
  static_assert(kSoftmaxRegs > kLaunchRegs && kOtherRegs < kLaunchRegs, "softmax takes more, the others give back");
  static_assert(2 * kSoftmaxRegs + (kProducers + 1) * kOtherRegs == kThreads / 128 * kLaunchRegs, "the block's registers");
};
constexpr float kTileLazy = 8.f;

template <int DP, bool E4>
struct Layout {
  static constexpr int kOp = kBlk * DP * 2;  // an operand tile: 128 rows, 64-column panels of 16 KB
  // Queries: row tiles in turn.  With a third place an item's first tile is there
  // before the item before is through; codes need that room for themselves.
  static constexpr int kQs = E4 ? 2 : 3;
  static constexpr int kQ = 0;
  static constexpr int kK = kQs * kOp;       // two buffers
  static constexpr int kV = kK + 2 * kOp;    // two buffers
  static constexpr int kStage = kV + 2 * kOp;        // codes: a block's keys and values as they are
  static constexpr int kCtrl = 7 * kOp;
  static constexpr int kSmem = kCtrl + 1024;
};

// One (row, block of 256 query rows, KV head, part of the keys), and what all
// roles have to know of it.
struct TileItem {
  int item;            // negative: there are no more
  int b, g, blk, split;
  int n, cnt;          // tokens before the pass; queries (negative: the row cannot be used)
  int r0;              // first query row
  int tiles;           // row tiles in use
  int end;             // keys lie below this token
  int p0, p1;          // the queries' positions lie in p0 .. p1
  int g0, g1;          // groups of keys
  int nblk;            // blocks of keys
};

constexpr int kItemSlots = 4;
constexpr int kOddSlots = 8;  // nobody is more than kItemSlots + 1 items ahead of another
struct TileCtrl {
  uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  uint64_t land[2], lfree[2];  // 16-bit values as they have come in (two places); codes of keys and of values
  uint64_t sfull[2], phalf[2], pfull[2], done[2], qfull[3], qfree[3], ofree[2], drain[2];
  uint64_t ifull[kItemSlots], ifree[kItemSlots];
  uint32_t tmem;
  int abort;
  // 1 + the item in which a value that is not finite was taken out, items with
  // keys in turn
  int odd[kOddSlots];
  TileItem items[kItemSlots];
};
static_assert(sizeof(TileCtrl) <= 1024, "control block");

__device__ __forceinline__ bool wait_on(TileCtrl *c, uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity, 10000)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity, 10000)) return true;
    if (*reinterpret_cast<volatile int *>(&c->abort)) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *reinterpret_cast<volatile int *>(&c->abort) = 1;
      return false;
    }
  }
}

__device__ __forceinline__ TileItem make_item(const PagedParams &P, int item, int blocks) {
  TileItem I;
  I.item = item;
  I.g = item % P.H;
  item /= P.H;
  I.split = item % P.splits;
  item /= P.splits;
  I.blk = blocks - 1 - item % blocks;  // the last block of a prompt sees most, so it comes first
  I.b = item / blocks;
  I.cnt = paged_queries(P, I.b, I.n);
  I.r0 = I.blk * 256;
  I.tiles = P.N * P.G - I.r0 > 128 ? 2 : 1;
  const int q_first = I.r0 / P.G, q_last = min((I.r0 + 255) / P.G, P.N - 1);
  const bool tree = P.W > 0;
  I.end = I.cnt <= q_first ? 0 : tree ? I.n + I.cnt : I.n + min(I.cnt, q_last + 1);
  I.p0 = tree ? I.n : I.n + q_first;
  I.p1 = tree ? I.n + I.cnt : I.n + q_last;
  const Keys keys(P, I.p0, I.end);
  I.g0 = 0;
  I.g1 = keys.n;
  if (P.splits > 1) {  // parts of whole blocks
    const int per = ((keys.n + P.splits - 1) / P.splits + kBlkGroups - 1) / kBlkGroups * kBlkGroups;
    I.g0 = min(keys.n, I.split * per);
    I.g1 = min(keys.n, I.g0 + per);
  }
  I.nblk = (I.g1 - I.g0 + kBlkGroups - 1) / kBlkGroups;
  return I;
}

// The it-th item, by all lanes of a warp; false: a wait ran out.
__device__ __forceinline__ bool take_item(TileCtrl *c, int it, TileItem &I, uint64_t limit) {
  const int s = it % kItemSlots;
  if (!__all_sync(FULL_MASK, wait_on(c, &c->ifull[s], (it / kItemSlots) & 1, limit))) return false;
  I = c->items[s];
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(&c->ifree[s]);
  return true;
}

// Whether some query at a position in p0 .. p1 does not see some token of the group.
__device__ __forceinline__ bool group_masked(const PagedParams &P, int t0, int n, int p0, int p1) {
  return t0 + kGroup - 1 > (P.W > 0 ? n - 1 : p0) || (t0 + kGroup > P.sinks && t0 < window_from(P, p1));
}

// Which of a group's 16 tokens a query sees (bits): at position p, its window's
// first token, the row's n tokens before the pass, and (trees) its words.
__device__ __forceinline__ uint32_t group_seen(const PagedParams &P, int t0, int p, int from, int n, int end, const uint32_t *anc) {
  auto below = [&](int t) {  // tokens of the group below t
    const int k = t - t0;
    return k <= 0 ? 0u : k >= 16 ? 0xffffu : (1u << k) - 1u;
  };
  uint32_t bits = below(anc ? min(n, end) : min(p + 1, end));
  bits &= ~below(from) | below(P.sinks);
  if (anc && t0 + kGroup > n) {
    const int j = t0 - n;  // the first token's index among the pass's own
    uint32_t own;
    if (j < 0) {
      own = __ldg(anc) << -j;
    } else {
      const int w = j >> 5;
      own = __funnelshift_r(w < P.W ? __ldg(anc + w) : 0u, w + 1 < P.W ? __ldg(anc + w + 1) : 0u, j & 31);
    }
    bits |= own & below(end) & ~below(n);
  }
  return bits;
}

// Four e4m3 codes as bf16 numbers times a power of two (all of it exact): a code's
// exponent and fraction are moved to where bf16 has them, which makes it 2^-120 of
// its value (its subnormal numbers are bf16's there), and multiplied up: at once
// by 2^120 and the scale where that is a bf16 number (scales up to 2^7), else in
// two steps.  A code of NaN comes out as 480 times the scale, which code_nan() tells.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t factor) {
  // a number's two bytes: sign and the code's upper bits, the code's lower bits
  const uint32_t up = ((w >> 4) & 0x07070707u) | (w & 0x80808080u), lo = (w * 16u) & 0xf0f0f0f0u;
  return make_uint2(mul_bf16x2(__byte_perm(lo, up, 0x5140), factor), mul_bf16x2(__byte_perm(lo, up, 0x7362), factor));
}
// Nonzero in the upper bit of every byte that is a code of NaN.
__device__ __forceinline__ uint32_t code_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint2 with_nans(uint2 r, uint32_t nan) {
  if (nan & 0x80u) r.x |= 0x7fc0u;
  if (nan & 0x8000u) r.x |= 0x7fc00000u;
  if (nan & 0x800000u) r.y |= 0x7fc0u;
  if (nan & 0x80000000u) r.y |= 0x7fc00000u;
  return r;
}
constexpr uint32_t kTopScale = 134;  // the largest scale byte that goes with 2^120 in one bf16 number
// 2^120 times the scale of byte c (of kTopScale, if c is larger), as a pair of bf16; NaN for 255
__device__ __forceinline__ uint32_t first_factor(uint32_t c) {
  const uint32_t h = c == 255u ? 0x7fc0u : (min(c, kTopScale) + 120u) << 7;
  return h | h << 16;
}
// the rest of the scale
__device__ __forceinline__ uint32_t second_factor(uint32_t c) {
  const uint32_t h = c == 255u || c <= kTopScale ? 0x3f80u : (c - kTopScale + 127u) << 7;
  return h | h << 16;
}

// Whether one of eight 16-bit numbers is an infinity or NaN; these set to zero.
template <bool BF>
__device__ __forceinline__ bool not_finite(const uint4 &u) {
  constexpr uint32_t top = BF ? 0x7f807f80u : 0x7c007c00u, one = BF ? 0x00800080u : 0x04000400u;
  return (((u.x & top) + one) | ((u.y & top) + one) | ((u.z & top) + one) | ((u.w & top) + one)) & 0x80008000u;
}
template <bool BF>
__device__ __forceinline__ void drop_not_finite(uint4 &u) {
  constexpr uint32_t top = BF ? 0x7f80u : 0x7c00u;
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((w[e] & top) == top) w[e] &= 0xffff0000u;
    if ((w[e] >> 16 & top) == top) w[e] &= 0x0000ffffu;
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight elements from any address; zeros if not `on`.
__device__ __noinline__ void copy_eight(unsigned char *to, const unsigned short *q, bool on) {
  uint32_t u[4] = {0, 0, 0, 0};
  if (on)
    for (int i = 0; i < 4; ++i) u[i] = q[2 * i] | static_cast<uint32_t>(q[2 * i + 1]) << 16;
  *reinterpret_cast<uint4 *>(to) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float max3f(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Where a row's keys lie: lane i of a warp knows groups i of four blocks, and asks for
// the next four blocks' pages two blocks ahead.
struct Pages {
  int page, token, first;  // page (one past the last: none), token in it, token of the row
  int next_page, next_token, next_first;
  __device__ __forceinline__ void ask(const PagedParams &P, const TileItem &I, const Keys &keys, int k, int lane) {
    const int i = I.g0 + k * kBlkGroups + lane;
    next_page = max(P.pages, 1);
    next_token = 0;
    next_first = 0x7fffff00;
    if (i < I.g1) {
      next_first = keys.token(i);
      const int j = next_first / P.page, pg = __ldg(P.table + static_cast<size_t>(I.b) * P.columns + j);
      next_token = next_first - j * P.page;
      if (pg >= 0 && pg < P.pages) next_page = pg;
    }
  }
  // before block k's groups are used
  __device__ __forceinline__ void step(const PagedParams &P, const TileItem &I, const Keys &keys, int k, int lane) {
    if (k % 4 == 0) {
      if (k == 0) ask(P, I, keys, 0, lane);
      page = next_page;
      token = next_token;
      first = next_first;
    }
    if (k % 4 == 2 && k + 2 < I.nblk) ask(P, I, keys, k + 2, lane);
  }
};

// Keys and values as [page][token][head][number], a box being 16 tokens of one head.
struct PagedMaps {
  CUtensorMap k, v;
};

template <int CT, int DP>
__global__ void __launch_bounds__(Team<CT == SPEC_E4M3>::kThreads, 1)
    paged_tile_kernel(const __grid_constant__ PagedParams P, const __grid_constant__ PagedMaps M, int blocks, int items) {
  using C = Layout<DP, CT == SPEC_E4M3>;
  constexpr bool E4 = CT == SPEC_E4M3, BF = CT != SPEC_F16;
  using T = Team<E4>;
  extern __shared__ __align__(1024) unsigned char smem[];
  TileCtrl *const c = reinterpret_cast<TileCtrl *>(smem + C::kCtrl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, role = tid / 128;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->kfull[i], E4 ? 128 : 1);
      mbar_init(&c->vfull[i], 128);
      mbar_init(&c->kfree[i], 2);
      mbar_init(&c->vfree[i], 2);
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->phalf[i], 128);
      mbar_init(&c->pfull[i], 128);
      mbar_init(&c->done[i], 1);
      mbar_init(&c->ofree[i], 128);
      mbar_init(&c->land[i], 1);
      mbar_init(&c->lfree[i], 128);
      mbar_init(&c->drain[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&c->qfull[i], 128);
      mbar_init(&c->qfree[i], 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(&c->ifull[i], 1);
      mbar_init(&c->ifree[i], T::kProducers * 4 + 2 + 1 + 8);  // warps: producers, issue, loads, softmax
    }
    for (int i = 0; i < kOddSlots; ++i) c->odd[i] = 0;
    c->abort = 0;
    fence_mbar_init();
  }
  if (warp == T::kIssueWarp) tc_alloc(&c->tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const uint64_t limit = P.wait_limit_ns;
  const bool tree = P.W > 0;

  if (role >= 2 && role < T::kRest) {
    // ------------------------------------------------------------ producers
    // (Of two warpgroups the first has keys and queries, the second values.)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(T::kOtherRegs));
    const int val = E4 ? role - 2 : 1, pt = tid % 128;
    bool live = true;
    // A thread deals with 16-byte pieces of every kStep-th token of a block.
    constexpr int L = E4 ? DP / 16 : DP / 8, kStep = 128 / L, kPer = kBlk / kStep;
    static_assert(!E4 || kPer == L, "a lane's piece is the number of the token whose scale it reads");
    const int pc = pt % L, row0 = pt / L;
    constexpr int kPut = E4 ? 2048 : kStep * 128;
    int kb = 0, worked = 0, nq = 0;  // blocks, items and row tiles so far
    const bool vec = reinterpret_cast<uintptr_t>(P.q) % 16 == 0 && P.qs[0] % 8 == 0 && P.qs[1] % 8 == 0 && P.qs[2] % 8 == 0;
    TileItem I;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (live) live = wait_on(c, bar, parity, limit);
      live = __all_sync(FULL_MASK, live);
    };
    for (int turn = 0; live && take_item(c, turn, I, limit) && I.item >= 0; ++turn) {
      if (I.nblk == 0) continue;
      const Keys keys(P, I.p0, I.end);
      // queries of a row tile: DP / 8 lanes per row, 16 bytes each, once the scores
      // of the place's former tile are done (all tiles' by the same warps: places are
      // waited for in order)
      auto hand_queries = [&]() {
        cp_async_wait_all();
        fence_async_smem();
        for (int t = nq - I.tiles; t < nq; ++t) mbar_arrive(&c->qfull[t % C::kQs]);
      };
#pragma unroll 1
      for (int tile = 0; tile < I.tiles && !(E4 && val); ++tile, ++nq) {
        constexpr int QL = DP / 8, kRows = 128 / QL;
        const int qc = pt % QL, place = nq % C::kQs;
        if (nq >= C::kQs) wait(&c->qfree[place], (nq / C::kQs - 1) & 1);
        if (!live) break;
        const int r = I.r0 + tile * 128 + pt / QL;
        int t = r / P.G, h = r - t * P.G;  // the row's token and head of the group
        const unsigned short *q = static_cast<const unsigned short *>(P.q) + I.b * P.qs[0] + t * P.qs[1] +
                                  (static_cast<long long>(I.g) * P.G + h) * P.qs[2] + qc * 8;
        unsigned char *to = smem + C::kQ + place * C::kOp + (qc / 8) * 16384 + (pt / QL) * 128 + (((qc % 8) ^ (pt / QL & 7)) << 4);
        const int dt = kRows / P.G, dh = kRows - dt * P.G;
        const long long step = dt * P.qs[1] + dh * P.qs[2], wrap = P.qs[1] - P.G * P.qs[2];
        const bool in = qc * 8 < P.D;
#pragma unroll 2
        for (int i = 0; i < 128 / kRows; ++i) {
          const bool on = in && t < P.N;
          if (vec)
            cp_async16_zfill(smem_u32(to), on ? q : static_cast<const unsigned short *>(P.q), on);
          else
            copy_eight(to, q, on);
          to += kRows * 128;
          t += dt;
          h += dh;
          q += step;
          if (h >= P.G) h -= P.G, ++t, q += wrap;
        }
        if (!E4) {  // the second tile's place may be a while in coming free
          cp_async_wait_all();
          fence_async_smem();
          mbar_arrive(&c->qfull[place]);
        }
      }
      if (!live) break;
      // In groups that some query does not see whole, values that are not finite
      // are taken out (it would get 0 * NaN) and put into the answers of the
      // queries that see them at the end; what lies behind the last token was
      // brought along, and is nobody's.
      auto partial = [&](int k) {  // such groups of the block
        const int gi = I.g0 + k * kBlkGroups + (lane & 7);
        return __ballot_sync(FULL_MASK, gi < I.g1 && group_masked(P, keys.token(gi), I.n, I.p0, I.p1)) & 0xffu;
      };
      auto behind = [&](int k, int row) { return keys.token(I.g0 + k * kBlkGroups + row / 16) + row % 16 >= I.end; };
      if constexpr (!E4) {
        for (int k = 0; k < I.nblk; ++k) {
          const int at = kb + k, s = at & 1;
          wait(&c->land[s], (at >> 1) & 1);
          if (!live) break;
          const unsigned part = partial(k);
          if (part) {
            unsigned char *const buf = smem + C::kV + s * C::kOp + (pc / 8) * 16384 + row0 * 128 + (((pc % 8) ^ (row0 & 7)) << 4);
            constexpr int kRun = kPer < 8 ? kPer : 8;
            bool some = false, odd = false;
#pragma unroll 1
            for (int i0 = 0; i0 < kPer; i0 += kRun) {
              uint4 w[kRun];
#pragma unroll
              for (int i = 0; i < kRun; ++i) w[i] = *reinterpret_cast<const uint4 *>(buf + (i0 + i) * kPut);
#pragma unroll
              for (int i = 0; i < kRun; ++i) some = some || not_finite<BF>(w[i]);
            }
            if (some) {
#pragma unroll 1
              for (int i = 0; i < kPer; ++i) {
                const int row = row0 + i * kStep;
                uint4 w = *reinterpret_cast<const uint4 *>(buf + i * kPut);
                if (!(part >> (row / 16) & 1u) || !not_finite<BF>(w)) continue;
                drop_not_finite<BF>(w);
                *reinterpret_cast<uint4 *>(buf + i * kPut) = w;
                odd = odd || !behind(k, row);
              }
            }
            if (odd) c->odd[worked % kOddSlots] = I.item + 1;
            fence_async_smem();
          }
          mbar_arrive(&c->vfull[s]);
        }
      } else {
        // Each thread's scale byte, of the block's token row0 + pc kStep, is asked for
        // a block ahead.
        Pages where;
        auto scale = [&](int k) -> uint32_t {
          uint32_t byte = 0;
          if (k < I.nblk) {
            const int row = row0 + pc * kStep, from = (k % 4) * kBlkGroups + row / 16;
            where.step(P, I, keys, k, lane);
            const int pg = __shfl_sync(FULL_MASK, where.page, from), t = __shfl_sync(FULL_MASK, where.token, from);
            const int first = __shfl_sync(FULL_MASK, where.first, from);
            if (pg < P.pages && first + row % 16 < I.end)
              byte = __ldg((val ? P.v : P.k) + pg * P.page_stride + (t + row % 16) * P.tok_stride + static_cast<long long>(P.H) * P.D + I.g);
          }
          return byte;
        };
        const unsigned char *const codes = smem + C::kStage + val * (C::kOp / 2) + pt * 16;
        uint32_t sc0 = scale(0);
        for (int k = 0; k < I.nblk; ++k) {
          const int at = kb + k, s = at & 1;
          const unsigned part = val ? partial(k) : 0;
          const uint32_t sc1 = scale(k + 1);
          wait(&c->land[val], at & 1);
          if (k == 0 && live && !val) hand_queries();
          if (at >= 2) wait(val ? &c->vfree[s] : &c->kfree[s], ((at >> 1) - 1) & 1);
          if (!live) break;
          unsigned char *const buf = smem + (val ? C::kV : C::kK) + s * C::kOp;
          bool odd = false;
          // (255 among them: a scale of NaN)
          const bool large = __any_sync(FULL_MASK, sc0 > kTopScale);
          const int ch = (pc % 4) * 2, up = pc / 4;
          uint32_t nans = 0;
#pragma unroll 2
          for (int i = 0; i < kPer; ++i) {
            const int row = row0 + i * kStep;
            uint4 w = *reinterpret_cast<const uint4 *>(codes + i * kPut);
            const uint32_t f = first_factor(__shfl_sync(FULL_MASK, sc0, (lane & ~(L - 1)) + i));
            nans |= code_nan(w.x) | code_nan(w.y) | code_nan(w.z) | code_nan(w.w);
            // the two 16-byte halves, the upper panel's lanes in the other
            // order: eight lanes then cover all banks
            if (up) w = make_uint4(w.z, w.w, w.x, w.y);
            const uint2 y0 = codes_to_bf16(w.x, f), y1 = codes_to_bf16(w.y, f), y2 = codes_to_bf16(w.z, f), y3 = codes_to_bf16(w.w, f);
            unsigned char *const to = buf + up * 16384 + row * 128;
            *reinterpret_cast<uint4 *>(to + (((ch + up) ^ (row & 7)) << 4)) = make_uint4(y0.x, y0.y, y1.x, y1.y);
            *reinterpret_cast<uint4 *>(to + (((ch + 1 - up) ^ (row & 7)) << 4)) = make_uint4(y2.x, y2.y, y3.x, y3.y);
          }
          // what is rare: large scales, codes and scales of NaN
          if (large || __any_sync(FULL_MASK, nans != 0)) {
#pragma unroll 1
            for (int i = 0; i < kPer; ++i) {
              const int row = row0 + i * kStep;
              const uint4 w = *reinterpret_cast<const uint4 *>(codes + i * kPut);
              const uint32_t c0 = __shfl_sync(FULL_MASK, sc0, (lane & ~(L - 1)) + i);
              const uint32_t f = first_factor(c0), f2 = second_factor(c0);
              uint32_t cw[4] = {w.x, w.y, w.z, w.w}, y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint2 z = codes_to_bf16(cw[e], f);
                z = with_nans(make_uint2(mul_bf16x2(z.x, f2), mul_bf16x2(z.y, f2)), code_nan(cw[e]));
                y[2 * e] = z.x, y[2 * e + 1] = z.y;
              }
              uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
              if ((part >> (row / 16) & 1u) && (not_finite<true>(lo) || not_finite<true>(hi))) {
                drop_not_finite<true>(lo);
                drop_not_finite<true>(hi);
                odd = odd || !behind(k, row);
              }
              unsigned char *const to = buf + up * 16384 + row * 128;
              *reinterpret_cast<uint4 *>(to + ((ch ^ (row & 7)) << 4)) = lo;
              *reinterpret_cast<uint4 *>(to + (((ch + 1) ^ (row & 7)) << 4)) = hi;
            }
          }
          mbar_arrive(&c->lfree[val]);
          if (odd) c->odd[worked % kOddSlots] = I.item + 1;
          fence_async_smem();
          mbar_arrive(val ? &c->vfull[s] : &c->kfull[s]);
          sc0 = sc1;
        }
      }
      kb += I.nblk;
      ++worked;
    }
    cp_async_wait_all();
  } else if (role == T::kRest) {
    // ------------------------------------------------- tensor-core issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(T::kOtherRegs));
    // A warp for each tile: the tensor cores take an instruction at a time from each
    // and hardly queue any, so that with one warp for both they stood still while it
    // waited (150 us a prompt, so 145).  All of a warp runs through this and one lane
    // does it, with operands that the compiler knows to be the same in all lanes.
    if (warp == T::kIssueWarp || warp == T::kIssueWarp + 1) {
      const int t = __shfl_sync(FULL_MASK, warp == T::kIssueWarp + 1, 0);
      const uint32_t qk = inst_desc(BF, kBlk, false), wv = inst_desc(BF, DP, true);
      const uint32_t base = __shfl_sync(FULL_MASK, smem_u32(smem), 0), tm = __shfl_sync(FULL_MASK, tmem, 0) + t * 128;
      const uint64_t qd = op_desc(base + C::kQ, 16), kd = op_desc(base + C::kK, 16), vd = op_desc(base + C::kV, 16384);
      bool live = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) { live = live && __all_sync(FULL_MASK, wait_on(c, bar, parity, limit)); };
      int kb = 0, nq = 0, ni = 0, nb = 0;  // blocks and row tiles in all; the tile's items and blocks
      for (int turn = 0; live; ++turn) {
        const int slot = turn % kItemSlots;
        wait(&c->ifull[slot], (turn / kItemSlots) & 1);
        if (!live) break;
        const int item = __shfl_sync(FULL_MASK, c->items[slot].item, 0);
        const int nblk = __shfl_sync(FULL_MASK, c->items[slot].nblk, 0), tiles = __shfl_sync(FULL_MASK, c->items[slot].tiles, 0);
        if (lane == 0) mbar_arrive(&c->ifree[slot]);
        if (item < 0) break;
        if (nblk == 0) continue;
        if (t < tiles) {
          const int place = (nq + t) % C::kQs;
          wait(&c->qfull[place], ((nq + t) / C::kQs) & 1);
          // block k's weights times values, then block k + 1's scores in their place
#pragma unroll 1
          for (int k = -1; k < nblk; ++k) {
            const int at = kb + k;
            if (k >= 0) {
              wait(&c->vfull[at & 1], (at >> 1) & 1);
              // the item before's answers have to be out of the sums
              if (k == 0 && ni > 0) wait(&c->ofree[t], (ni - 1) & 1);
              // the first half's product runs while the second half's weights are made
              // (a prompt 148 us without, 142 with)
              wait(&c->phalf[t], (nb + k) & 1);
              if (!live) break;
              const uint64_t bb = vd + static_cast<uint32_t>((at & 1) * C::kOp >> 4);
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int j = 0; j < kBlk / 32; ++j) tc_mma_ts(tm + 256, tm + j * 8, bb + (j * 2048 >> 4), wv, k > 0 || j > 0);
              }
              wait(&c->pfull[t], (nb + k) & 1);
              if (!live) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int j = kBlk / 32; j < kBlk / 16; ++j) tc_mma_ts(tm + 256, tm + j * 8, bb + (j * 2048 >> 4), wv, true);
                tc_commit(&c->vfree[at & 1]);
                if (k + 1 == nblk) tc_commit(&c->done[t]);
              }
              if (k + 1 == nblk) break;
            }
            wait(&c->kfull[(at + 1) & 1], ((at + 1) >> 1) & 1);
            if (!live) break;
            const uint64_t a = qd + static_cast<uint32_t>(place * C::kOp >> 4), bb = kd + static_cast<uint32_t>(((at + 1) & 1) * C::kOp >> 4);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int d = 0; d < DP / 16; ++d) {
                const int off = ((d / 4) * 16384 + (d % 4) * 32) >> 4;
                tc_mma_ss(tm, a + off, bb + off, qk, d > 0);
              }
              tc_commit(&c->sfull[t]);
              tc_commit(&c->kfree[(at + 1) & 1]);
              if (k + 2 == nblk) tc_commit(&c->qfree[place]);  // the tile's last
            }
          }
          ++ni;
          nb += nblk;
        } else {
          // The tile's warp goes through the blocks all the same: neither warp may be
          // two of a buffer's turns ahead, where one turn looks like the other.
          for (int k = 0; k < nblk && live; ++k) {
            const int at = kb + k;
            wait(&c->kfull[at & 1], (at >> 1) & 1);
            if (live && lane == 0) mbar_arrive(&c->kfree[at & 1]);
            wait(&c->vfull[at & 1], (at >> 1) & 1);
            if (live && lane == 0) mbar_arrive(&c->vfree[at & 1]);
          }
        }
        kb += nblk;
        nq += tiles;
      }
      if (!live) {  // let what was issued end before tensor memory is given back
        if (elect_one()) tc_commit(&c->drain[t]);
        mbar_wait_bounded(&c->drain[t], 0, limit);
      }
    } else if (warp == T::kLoadWarp) {
      // ------------------------------------------- keys and values on their way
      bool live = true;
      int kb = 0;
      uint32_t brought[2] = {0, 0};  // times so far: keys, values
      TileItem I;
      for (int turn = 0; live && take_item(c, turn, I, limit) && I.item >= 0; ++turn) {
        const Keys keys(P, I.p0, I.end);
        Pages where;
        for (int it = 0; it < 2 * I.nblk; ++it) {
          const int k = it >> 1, at = kb + k, s = at & 1;
          const bool val = it & 1;
          if (!val) where.step(P, I, keys, k, lane);
          // codes: the place of keys or of values once it has been read; 16-bit entries:
          // a block's
          if constexpr (E4) {
            if (at >= 1) live = __all_sync(FULL_MASK, wait_on(c, &c->lfree[val], (at - 1) & 1, limit));
          } else {
            if (at >= 2) live = __all_sync(FULL_MASK, wait_on(c, val ? &c->vfree[s] : &c->kfree[s], ((at >> 1) - 1) & 1, limit));
          }
          if (!live || (it == 0 && (P.force_timeout == 1 || P.force_timeout == I.g + 2))) {
            live = false;
            break;
          }
          uint64_t *const bar = E4 ? &c->land[val] : val ? &c->land[s] : &c->kfull[s];
          const uint32_t to = smem_u32(smem) + (E4 ? C::kStage + val * (C::kOp / 2) : (val ? C::kV : C::kK) + s * C::kOp);
          const CUtensorMap *const map = val ? &M.v : &M.k;
          if (elect_one()) mbar_arrive_expect_tx(bar, E4 ? C::kOp / 2 : C::kOp);
          __syncwarp();
#pragma unroll 1
          for (int j = 0; j < kBlkGroups; ++j) {
            const int pg = __shfl_sync(FULL_MASK, where.page, (k % 4) * kBlkGroups + j), t = __shfl_sync(FULL_MASK, where.token, (k % 4) * kBlkGroups + j);
            if (elect_one()) {
              if constexpr (E4) {
                tma_load_4d(to + j * kGroup * DP, map, 0, I.g, t, pg, bar);
              } else {
#pragma unroll
                for (int x = 0; x < DP; x += 64) tma_load_4d(to + x / 64 * 16384 + j * kGroup * 128, map, x, I.g, t, pg, bar);
              }
            }
          }
          ++brought[val];
        }
        kb += I.nblk;
      }
      // Nothing may come in behind the block's end, if a wait of whichever warp ran
      // out: each place's last boxes are waited for (and of no phase but a barrier's
      // last: one before it would count as still to come).
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        constexpr uint32_t kPlaces = E4 ? 1 : 2;
        for (uint32_t n = brought[i] > kPlaces ? brought[i] - kPlaces : 0; n < brought[i]; ++n) {
          if constexpr (E4)
            mbar_wait_bounded(&c->land[i], n & 1, limit);
          else
            mbar_wait_bounded(i ? &c->land[n & 1] : &c->kfull[n & 1], (n >> 1) & 1, limit);
        }
      }
    } else if (warp == T::kItemWarp) {
      // ------------------------------------------------------------- items
      if (lane == 0) {
        bool live = true;
        for (int turn = 0, item = blockIdx.x; live; ++turn, item += gridDim.x) {
          const int slot = turn % kItemSlots;
          TileItem I;
          if (item < items)
            I = make_item(P, item, blocks);
          else
            I.item = -1;
          if (turn >= kItemSlots) live = wait_on(c, &c->ifree[slot], (turn / kItemSlots - 1) & 1, limit);
          if (!live) break;
          c->items[slot] = I;
          mbar_arrive(&c->ifull[slot]);
          if (item >= items) break;
        }
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(T::kSoftmaxRegs));
    const int tile = role, rr = tid;  // tile and row of the block: tile * 128 + lane of tensor memory
    const int wt = tid % 128;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t s_addr = lane_addr + tile * 128, o_addr = lane_addr + 256 + tile * 128;
    const float sc = fmaxf(fabsf(P.scale), 0x1p-149f);  // not zero: a key that is not seen has the score -inf (what is seen stays below 2^-21)
    const bool minus = P.scale < 0.f, sectors = reinterpret_cast<uintptr_t>(P.out) % 32 == 0;
    bool live = true, checked = false;
    int worked = 0;  // items with keys
    uint32_t ni = 0, nb = 0;  // the tile's items and blocks so far
    if (tree) grid_dependency_wait();
    TileItem next;
    next.tiles = next.nblk = 0;
    next.item = next.b = next.g = next.blk = next.split = next.n = next.cnt = next.r0 = next.end = next.p0 = next.p1 = next.g0 = next.g1 = 0;
    struct Row {
      int at, my;     // the thread's output row (-1: past the last) and token
      int p, p0, p1;  // its position; the warp's rows' lie in p0 .. p1
      bool use;
    } row = {-1, 0, 0, 0, 0, false};
    for (int turn = -1; next.item >= 0; ++turn) {
      const TileItem I = next;
      const int at = row.at, my = row.my, p = row.p, p0 = row.p0, p1 = row.p1;
      const bool use = row.use;
      const int slot = worked % kOddSlots;
      worked += I.nblk > 0;
      const bool here = tile < I.tiles, work = here && I.nblk > 0 && live;
      const long long ml_at = static_cast<long long>(I.split) * P.rows + at;
      const long long flag = ((static_cast<long long>(I.b) * P.H + I.g) * blocks + I.blk) * P.splits + I.split;
      unsigned short *const answer = static_cast<unsigned short *>(P.out) + static_cast<long long>(at) * P.D;
      auto empty = [&](bool timeout) {
        if (at < 0) return;
        if (P.splits > 1) {
          P.ml[ml_at] = make_float2(-INFINITY, timeout ? __uint_as_float(kTimeoutBits) : -INFINITY);
          return;
        }
        for (int d = 0; d < P.D; d += 8) *reinterpret_cast<uint4 *>(answer + d) = make_uint4(0, 0, 0, 0);
        if (P.lse) P.lse[at] = -INFINITY;
        if (timeout && P.row_status) P.row_status[I.b] = SPEC_ROW_TIMEOUT;
      };
      if (here && !work) {
        if (wt == 0 && tile == 0 && P.splits > 1) P.oflag[flag] = 0;
        if (!checked) grid_dependency_wait();  // the status may not come before the check's
        checked = true;
        empty(I.nblk > 0);
      }
      const int from = window_from(P, p);
      const uint32_t *const anc = tree ? P.anc + (static_cast<size_t>(I.b) * P.N + my) * P.W : nullptr;
      const Keys keys(P, I.p0, I.end);
      float m = -INFINITY, l = 0.f;
      for (int k = 0; work && k < I.nblk; ++k) {
        // Groups of the block that some query of the warp does not see whole: what is
        // not seen gets the score -inf, in tensor memory and ahead of the rest, so
        // that this code, which most blocks pass by, stays out of the loop's way (the
        // roles' loops together just fit the instruction cache).
        unsigned part;
        {
          const int gi = I.g0 + k * kBlkGroups + (lane & 7);
          part = __ballot_sync(FULL_MASK, gi >= I.g1 || group_masked(P, keys.token(gi), I.n, p0, p1)) & 0xffu;
        }
        uint32_t b0 = 0, b1 = 0, b2 = 0, b3 = 0;  // (made while the scores are)
        if (part) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t bits = 0xffffffffu;
            if (part >> (2 * q) & 3u) {
              bits = 0;
#pragma unroll 1
              for (int j = 0; j < 2; ++j) {
                const int gi = I.g0 + k * kBlkGroups + 2 * q + j;
                if (gi < I.g1) bits |= group_seen(P, keys.token(gi), p, from, I.n, I.end, anc) << (16 * j);
              }
            }
            b0 = b1, b1 = b2, b2 = b3, b3 = ~bits;
          }
        }
        live = __all_sync(FULL_MASK, wait_on(c, &c->sfull[tile], (nb + k) & 1, limit));
        if (!live) break;
        tc_fence_after();
        if (part || minus) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const uint32_t bits = b0;
            b0 = b1, b1 = b2, b2 = b3;
            if (__all_sync(FULL_MASK, bits == 0u) && !minus) continue;
            uint32_t x[32];
            tc_ld32(x, s_addr + q * 32);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = bits >> j & 1 ? 0xff800000u : minus ? x[j] ^ 0x80000000u : x[j];
            tc_st32(s_addr + q * 32, x);
          }
          tc_wait_st();
        }
        auto largest = [](const uint32_t (&x)[32]) {
          float y = __uint_as_float(x[0]), z = __uint_as_float(x[1]);
#pragma unroll
          for (int j = 2; j < 30; j += 4) {
            y = max3f(y, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
            z = max3f(z, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
          }
          return fmaxf(max3f(y, __uint_as_float(x[30]), __uint_as_float(x[31])), z);
        };
        // 64 of the row's 128 scores are held at a time (all of them do not fit
        // in registers beside the rest): the upper half is read for the maximum,
        // then the lower half, whose weights are taken first, then the upper
        // half again.
        uint32_t s[2][32];
        float mq[4];
        tc_ld32(s[0], s_addr + 64);
        tc_ld32(s[1], s_addr + 96);
        tc_wait_ld();
        mq[2] = largest(s[0]);
        mq[3] = largest(s[1]);
        tc_ld32(s[0], s_addr);
        tc_ld32(s[1], s_addr + 32);
        tc_wait_ld();
        mq[0] = largest(s[0]);
        mq[1] = largest(s[1]);
        const float mt = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sc;
        float al = 1.f;
        if (mt > m + kTileLazy || m == -INFINITY) {
          al = mt == -INFINITY ? 1.f : ex2(m - mt);
          m = mt;
        }
        if (k > 0 && __any_sync(FULL_MASK, al != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < DP / 32; ++q) {
            uint32_t o[32];
            tc_ld32(o, o_addr + q * 32);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
            tc_st32(o_addr + q * 32, o);
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 sc2 = make_float2(sc, sc), off2 = make_float2(-ref, -ref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weights = [&](const uint32_t (&x)[32], int q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = ffma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sc2, off2);
            const float2 w = make_float2(ex2(y.x), ex2(y.y));
            sum[j & 1] = fadd2(sum[j & 1], w);
            pk[j] = pack16<BF>(w.x, w.y);
          }
          tc_st16(s_addr + q * 16, pk);  // over scores of the lower half, which have been read
        };
        weights(s[0], 0);
        tc_ld32(s[0], s_addr + 64);
        weights(s[1], 1);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c->phalf[tile]);
        tc_wait_ld();
        tc_ld32(s[1], s_addr + 96);
        weights(s[0], 2);
        tc_wait_ld();
        weights(s[1], 3);
        l = fmaf(l, al, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c->pfull[tile]);
      }
      // the next item, while the last product is made
      if (live) live = take_item(c, turn + 1, next, limit);
      if (!live) {  // what is left is empty, too
        const int item = blockIdx.x + (turn + 1) * gridDim.x;
        next.item = -1;
        if (item < items) next = make_item(P, item, blocks);
      }
      {
        const int r = next.r0 + rr;
        row.at = -1;
        row.my = 0;
        if (r < P.N * P.G) {
          row.my = r / P.G;
          row.at = (next.b * P.N + row.my) * P.Hq + next.g * P.G + (r - row.my * P.G);
        }
        row.use = next.item >= 0 && row.at >= 0 && row.my < next.cnt;
        const int q_first = min((r & ~31) / P.G, P.N - 1), q_last = min((r | 31) / P.G, P.N - 1);
        row.p = next.n + row.my;
        row.p0 = next.n + q_first;
        row.p1 = next.n + q_last;
        if (tree) {  // (a row that cannot be used has no depths: whatever stands there is not used)
          const int info = row.use ? P.rowinfo[next.b] : -1, d = row.use ? P.depth[static_cast<size_t>(next.b) * P.N + row.my] : 0;
          row.p = next.n + (info >= 0 ? d : 0);
          row.p0 = next.p0;
          row.p1 = next.p1;
        }
      }
      if (!work) continue;
      nb += I.nblk;
      if (!checked) grid_dependency_wait();  // the row's check
      checked = true;
      const bool some = use && P.rowinfo[I.b] >= 0 && l != 0.f;
      const float z = some ? m + log2f(l) : -INFINITY;
      if (live) live = __all_sync(FULL_MASK, wait_on(c, &c->done[tile], ni & 1, limit));
      ++ni;
      if (!live) {
        empty(true);
        if (wt == 0 && tile == 0 && P.splits > 1) P.oflag[flag] = 0;
        continue;
      }
      tc_fence_after();
      const bool odd = *reinterpret_cast<volatile int *>(&c->odd[slot]) == I.item + 1;
      const bool split = P.splits > 1;
      const float w = split ? 1.f : some ? ex2(m - z) : 0.f;
      float *const to = P.part + ml_at * P.D;
      if (split) {
        if (wt == 0 && tile == 0) P.oflag[flag] = odd;
        if (at >= 0) P.ml[ml_at] = some ? make_float2(m, z) : make_float2(-INFINITY, -INFINITY);
      } else if (at >= 0 && P.lse) {
        P.lse[at] = kLn2 * z;
      }
#pragma unroll 1
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t o[32];
        __syncwarp();
        tc_ld32(o, o_addr + q * 32);
        tc_wait_ld();
        if (q == DP / 32 - 1) {  // the sums are all read
          tc_fence_before();
          mbar_arrive(&c->ofree[tile]);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 16) {  // head sizes are multiples of 16: whole sectors
          if (q * 32 + j >= P.D) continue;
          if (split) {
            if (some) {
              st_global_v8(to + q * 32 + j, o + j);
              st_global_v8(to + q * 32 + j + 8, o + j + 8);
            }
          } else if (at >= 0) {
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              y[e] = some ? pack16<BF>(__uint_as_float(o[j + 2 * e]) * w, __uint_as_float(o[j + 2 * e + 1]) * w) : 0u;
            if (sectors) {
              st_global_v8(reinterpret_cast<float *>(answer + q * 32 + j), y);
            } else {
              *reinterpret_cast<uint4 *>(answer + q * 32 + j) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4 *>(answer + q * 32 + j + 8) = make_uint4(y[4], y[5], y[6], y[7]);
            }
          }
        }
      }
      if (odd && some && !split) {
        using N = typename CacheType<BF ? SPEC_BF16 : SPEC_F16>::type;
#pragma unroll 1
        for (int d = 0; d < P.D; ++d) {
          N *const y = reinterpret_cast<N *>(answer) + d;
          *y = N(static_cast<float>(*y) + paged_odd_sum<CT>(P, I.b, my, I.cnt, I.n, p, I.g, d));
        }
      }
    }
  }
  __syncthreads();
  grid_dependency_wait();
  if (warp == T::kIssueWarp) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem);
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess || r != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

template <int CT, int DP>
cudaError_t launch(const PagedParams &p, cudaStream_t s) {
  constexpr bool E4 = CT == SPEC_E4M3;
  using C = Layout<DP, E4>;
  const int blocks = (p.N * p.G + 255) / 256;
  const long long items = static_cast<long long>(p.B) * p.H * blocks * p.splits;
  if (items > 0x7fffffffLL - 4096) return cudaErrorInvalidValue;
  static_assert(C::kSmem <= 227 * 1024, "shared memory of a block");
  cudaError_t e = allow_smem<paged_tile_kernel<CT, DP>>(C::kSmem, Team<E4>::kLaunchRegs);
  if (e != cudaSuccess) return e;
  const EncodeTiled encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  PagedMaps m;
  const cuuint64_t pages = p.pages > 0 ? p.pages : 1;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.D), static_cast<cuuint64_t>(p.H), static_cast<cuuint64_t>(p.page), pages};
  // (the step between pages is not used where there is but one)
  const cuuint64_t steps[3] = {static_cast<cuuint64_t>(p.D) * (E4 ? 1 : 2), static_cast<cuuint64_t>(p.tok_stride),
                               static_cast<cuuint64_t>(pages > 1 ? p.page_stride : 16)};
  const cuuint32_t box[4] = {E4 ? DP : 64, 1, kGroup, 1}, ones[4] = {1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(i ? &m.v : &m.k, E4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<unsigned char *>(i ? p.v : p.k), dims,
               steps, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, E4 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
               E4 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(items < kPagedSms ? items : kPagedSms);
  return launch_after(paged_tile_kernel<CT, DP>, dim3(grid), Team<E4>::kThreads, C::kSmem, s, true, p, m, blocks, static_cast<int>(items));
}

template <int CT>
cudaError_t launch_d(const PagedParams &p, cudaStream_t s) {
  return p.D <= 64 ? launch<CT, 64>(p, s) : launch<CT, 128>(p, s);
}

}  // namespace

cudaError_t launch_paged_tile(const PagedParams &p, int ctype, cudaStream_t s) {
  if (ctype == SPEC_E4M3) return launch_d<SPEC_E4M3>(p, s);
  if (ctype == SPEC_BF16) return launch_d<SPEC_BF16>(p, s);
  return launch_d<SPEC_F16>(p, s);
}

}  // namespace sv
