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
//   - a block is eight groups of 16 keys, each from a page of its own: the
//     producers look eight addresses up at a time;
//   - e4m3 codes become bf16 numbers, scale and all, on their way into shared
//     memory.  That is exact (4 bits of significand, and bf16 has fp32's
//     exponents), so scales may lie any distance apart;
//   - a CTA runs through many items (a prompt has hundreds of them), and the
//     roles do not meet between them: a warpgroup loads its next queries as soon
//     as its last scores are in, the tensor cores start on them while it writes
//     the answers, and the producers run on through the pages.
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
constexpr int kTileThreads = 512;       // softmax of tiles A and B, producers, tensor-core issue
constexpr int kIssueWarp = 12;
constexpr int kLaunchRegs = 128;        // 65536 / kTileThreads
template <bool E4>
struct Regs {
  static constexpr int kSoftmax = E4 ? 176 : 184, kProduce = E4 ? 88 : 72, kIssue = 72;
  static_assert(kSoftmax > kLaunchRegs && kProduce < kLaunchRegs && kIssue < kLaunchRegs, "softmax takes more, the others give back");
  static_assert(2 * kSoftmax + kProduce + kIssue == 4 * kLaunchRegs, "the block's registers");
};
constexpr float kTileLazy = 8.f;

template <int DP>
struct Layout {
  static constexpr int kOp = kBlk * DP * 2;  // an operand tile: 128 rows, 64-column panels of 16 KB
  static constexpr int kQ = 0;               // tiles A and B
  static constexpr int kK = 2 * kOp;         // two buffers
  static constexpr int kV = 4 * kOp;         // two buffers
  static constexpr int kCtrl = 6 * kOp;
  static constexpr int kSmem = kCtrl + 4096 + 1024;  // + control block + alignment
};

struct TileCtrl {
  uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  uint64_t sfull[2], pfull[2], done[2], qfull[2], ofree[2], drain;
  uint32_t tmem;
  int abort;
  // 1 + the item in which a value that is not finite was taken out, four items
  // in turn (the producers are at most two blocks ahead of the tensor cores)
  int odd[4];
  uint32_t factor[2][kBlk];   // codes: the tokens' scales, keys and values
  int qoff[256][2];           // where a query row's elements are (two halves of 64 bits); -1: past the last
};
static_assert(sizeof(TileCtrl) <= 4096, "control block");

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

// One (row, block of 256 query rows, KV head, part of the keys), and what all
// roles have to know of it.
struct TileItem {
  int b, g, blk, split;
  int n, cnt;          // tokens before the pass; queries (negative: the row cannot be used)
  int r0;              // first query row
  int tiles;           // row tiles in use
  int end;             // keys lie below this token
  int p0, p1;          // the queries' positions lie in p0 .. p1
  int g0, g1;          // groups of keys
  int nblk;            // blocks of keys
  __device__ __forceinline__ TileItem(const PagedParams &P, int item, int blocks) {
    g = item % P.H;
    item /= P.H;
    split = item % P.splits;
    item /= P.splits;
    blk = blocks - 1 - item % blocks;  // the last block of a prompt sees most, so it comes first
    b = item / blocks;
    cnt = paged_queries(P, b, n);
    r0 = blk * 256;
    const int left = P.N * P.G - r0;
    tiles = left > 128 ? 2 : 1;
    const int q_first = r0 / P.G, q_last = min((r0 + 255) / P.G, P.N - 1);
    const bool tree = P.W > 0;
    end = cnt <= q_first ? 0 : tree ? n + cnt : n + min(cnt, q_last + 1);
    p0 = tree ? n : n + q_first;
    p1 = tree ? n + cnt : n + q_last;
    const Keys keys(P, p0, end);
    g0 = 0;
    g1 = keys.n;
    if (P.splits > 1) {  // parts of whole blocks
      const int per = ((keys.n + P.splits - 1) / P.splits + kBlkGroups - 1) / kBlkGroups * kBlkGroups;
      g0 = min(keys.n, split * per);
      g1 = min(keys.n, g0 + per);
    }
    nblk = (g1 - g0 + kBlkGroups - 1) / kBlkGroups;
  }
};

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
// its value (its subnormal numbers are bf16's there), and multiplied up.
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); }
__device__ __forceinline__ uint32_t from_bf2(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t factor) {
  const uint32_t lo = __byte_perm(w, 0, 0x1404), hi = __byte_perm(w, 0, 0x3424);
  const __nv_bfloat162 up = as_bf2(0x7b807b80u);  // 2^120
  const __nv_bfloat162 a = __hmul2(as_bf2((lo & 0x80008000u) | ((lo >> 4) & 0x07f007f0u)), up);
  const __nv_bfloat162 b = __hmul2(as_bf2((hi & 0x80008000u) | ((hi >> 4) & 0x07f007f0u)), up);
  uint2 r = make_uint2(from_bf2(__hmul2(a, as_bf2(factor))), from_bf2(__hmul2(b, as_bf2(factor))));
  if (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) {  // codes of NaN
    if ((w & 0x7fu) == 0x7fu) r.x |= 0x7fc0u;
    if ((w & 0x7f00u) == 0x7f00u) r.x |= 0x7fc00000u;
    if ((w & 0x7f0000u) == 0x7f0000u) r.y |= 0x7fc0u;
    if ((w & 0x7f000000u) == 0x7f000000u) r.y |= 0x7fc00000u;
  }
  return r;
}
// 2^(c - 127) as a pair of bf16; NaN for 255
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t c) {
  const uint32_t h = c == 255u ? 0x7fc0u : c ? c << 7 : 0x0040u;
  return h | h << 16;
}

__device__ __forceinline__ float max3f(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <int CT, int DP>
__global__ void __launch_bounds__(kTileThreads, 1) paged_tile_kernel(const __grid_constant__ PagedParams P, int blocks, int items) {
  using C = Layout<DP>;
  constexpr bool E4 = CT == SPEC_E4M3, BF = CT != SPEC_F16;
  using R = Regs<E4>;
  extern __shared__ unsigned char raw[];
  unsigned char *const smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  TileCtrl *const c = reinterpret_cast<TileCtrl *>(smem + C::kCtrl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, role = tid / 128;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->kfull[i], 128);
      mbar_init(&c->vfull[i], 128);
      mbar_init(&c->kfree[i], 1);
      mbar_init(&c->vfree[i], 1);
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->pfull[i], 128);
      mbar_init(&c->done[i], 1);
      mbar_init(&c->qfull[i], 128);
      mbar_init(&c->ofree[i], 128);
      c->odd[i] = c->odd[i + 2] = 0;
    }
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) tc_alloc(&c->tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const uint64_t limit = P.wait_limit_ns;
  const bool tree = P.W > 0;

  if (role == 2) {
    // ------------------------------------------------------------ producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kProduce));
    const int pt = tid - 256;
    bool live = true;
    // A thread brings 16-byte pieces of every kStep-th token of a block.
    constexpr int L = E4 ? DP / 16 : DP / 8, kStep = 128 / L, kPer = kBlk / kStep;
    const int pc = pt % L, row0 = pt / L;
    const bool col = pc * 16 < P.D * (E4 ? 1 : 2);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t put0 = E4 ? pt * 16 : (pc / 8) * 16384 + row0 * 128 + (((pc % 8) ^ (row0 & 7)) << 4);
    constexpr int kPut = E4 ? 2048 : kStep * 128;
    int kb = 0;     // blocks handed over so far
    int odd_at = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      const TileItem I(P, item, blocks);
      if (I.nblk == 0) continue;
      const Keys keys(P, I.p0, I.end);
      const int32_t *const trow = P.table + static_cast<size_t>(I.b) * P.columns;
      const long long piece = static_cast<long long>(I.g) * P.D * (E4 ? 1 : 2) + (col ? pc * 16 : 0);
      // lane i: where group i of four blocks starts in its plane (-1: on no page), and its first token
      long long where = -1;
      int first = 0;
      auto look_up = [&](int k) {
        const int i = I.g0 + k * kBlkGroups + lane;
        where = -1;
        first = 0;
        if (i < I.g1) {
          first = keys.token(i);
          const int j = first / P.page, pg = __ldg(trow + j);
          if (pg >= 0 && pg < P.pages) where = pg * P.page_stride + (first - j * P.page) * P.tok_stride;
        }
      };
      // copies of block k's keys or values; codes: the scale byte of the block's token pt
      auto issue = [&](int it) -> uint32_t {
        uint32_t byte = 0;
        if (it < 2 * I.nblk) {
          const int k = it >> 1, at = kb + k, s = at & 1;
          const bool val = it & 1;
          if (!val && k % 4 == 0) look_up(k);
          const int base = (k % 4) * kBlkGroups;
          const unsigned char *const plane = val ? P.v : P.k;
          if constexpr (E4) {
            const long long w = __shfl_sync(FULL_MASK, where, base + pt / 16);
            const int t = __shfl_sync(FULL_MASK, first, base + pt / 16) + pt % 16;
            if (w >= 0 && t < I.end) byte = __ldg(plane + w + pt % 16 * P.tok_stride + static_cast<long long>(P.H) * P.D + I.g);
          }
          if (at >= 2 && live) live = wait_on(c, val ? &c->vfree[s] : &c->kfree[s], ((at >> 1) - 1) & 1, limit);
          live = __all_sync(FULL_MASK, live);
          if (live) {
            const uint32_t dst = sbase + put0 + (val ? C::kV : C::kK) + s * C::kOp;
            constexpr int kSame = kStep < 16 ? 16 / kStep : 1;  // neighbouring copies in one group
#pragma unroll
            for (int i0 = 0; i0 < kPer; i0 += kSame) {
              const int row = row0 + i0 * kStep;
              const long long w = __shfl_sync(FULL_MASK, where, base + row / 16);
              const int t0 = __shfl_sync(FULL_MASK, first, base + row / 16);  // by every lane
              const int left = w < 0 || !col ? 0 : I.end - t0;
              const unsigned char *const src = plane + w + row % 16 * P.tok_stride + piece;
#pragma unroll
              for (int i = i0; i < i0 + kSame; ++i) {
                const bool on = row % 16 + (i - i0) * kStep < left;
                cp_async16_zfill(dst + i * kPut, on ? src + (i - i0) * kStep * P.tok_stride : plane, on);
              }
            }
          }
        }
        cp_async_commit();
        return byte;
      };
      uint32_t sc0 = issue(0), sc1 = issue(1);
      for (int it = 0; it < 2 * I.nblk; ++it) {
        cp_async_wait<1>();
        const int k = it >> 1, at = kb + k, s = at & 1;
        const bool val = it & 1;
        // In groups that some query does not see whole, values that are not
        // finite are taken out (it would get 0 * NaN) and put into the answers of
        // the queries that see them at the end.
        unsigned part = 0;  // such groups of the block
        if (val) {
#pragma unroll
          for (int i = 0; i < kBlkGroups; ++i) {
            const int gi = I.g0 + k * kBlkGroups + i;
            if (gi < I.g1 && group_masked(P, keys.token(gi), I.n, I.p0, I.p1)) part |= 1u << i;
          }
        }
        const uint32_t buf = sbase + (val ? C::kV : C::kK) + s * C::kOp;
        if constexpr (!E4) {
          if (part && live) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const int row = row0 + i * kStep;
              if (!(part >> (row / 16) & 1u)) continue;
              const uint32_t to = buf + put0 + i * kPut;
              uint32_t w[4];
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(to) : "memory");
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                constexpr uint32_t top = BF ? 0x7f80u : 0x7c00u;
                if ((w[e] & top) == top) w[e] &= 0xffff0000u, odd = true;
                if ((w[e] >> 16 & top) == top) w[e] &= 0x0000ffffu, odd = true;
              }
              if (odd) {
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
                c->odd[odd_at & 3] = item + 1;
              }
            }
          }
        } else {
          uint32_t w[kPer][4];
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                         : "r"(buf + put0 + i * kPut)
                         : "memory");
          c->factor[it & 1][pt] = scale_bf16x2(sc0);
          asm volatile("bar.sync 1, 128;" ::: "memory");  // every code has been read, every scale is there
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int row = row0 + i * kStep;
            const uint32_t f = c->factor[it & 1][row];
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 y = codes_to_bf16(w[i][e], f);
              o[2 * e] = y.x;
              o[2 * e + 1] = y.y;
            }
            if (part >> (row / 16) & 1u) {
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if ((o[e] & 0x7f80u) == 0x7f80u) o[e] &= 0xffff0000u, odd = true;
                if ((o[e] >> 16 & 0x7f80u) == 0x7f80u) o[e] &= 0x0000ffffu, odd = true;
              }
              if (odd) c->odd[odd_at & 3] = item + 1;
            }
            // the two 16-byte halves, the upper panel's lanes in the other
            // order: eight lanes then cover all banks
            const int ch = (pc % 4) * 2, up = pc / 4;
            const uint32_t to = buf + up * 16384 + row * 128;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((ch + up) ^ (row & 7)) << 4)),
                         "r"(up ? o[4] : o[0]), "r"(up ? o[5] : o[1]), "r"(up ? o[6] : o[2]), "r"(up ? o[7] : o[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((ch + 1 - up) ^ (row & 7)) << 4)),
                         "r"(up ? o[0] : o[4]), "r"(up ? o[1] : o[5]), "r"(up ? o[2] : o[6]), "r"(up ? o[3] : o[7])
                         : "memory");
          }
        }
        fence_async_smem();
        if (!(it == 0 && (P.force_timeout == 1 || P.force_timeout == I.g + 2))) mbar_arrive(val ? &c->vfull[s] : &c->kfull[s]);
        sc0 = sc1;
        sc1 = issue(it + 2);  // after this one is handed over: its buffer may be a while in coming free
      }
      kb += I.nblk;
      ++odd_at;
    }
    cp_async_wait_all();
  } else if (role == 3) {
    // ------------------------------------------------- tensor-core issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kIssue));
    if (warp == kIssueWarp && lane == 0) {
      const uint32_t qk = inst_desc(BF, kBlk, false), wv = inst_desc(BF, DP, true);
      const uint32_t base = smem_u32(smem);
      const uint64_t qd = op_desc(base + C::kQ, 16), kd = op_desc(base + C::kK, 16), vd = op_desc(base + C::kV, 16384);
      auto scores = [&](int tile, int at) {
        const uint64_t a = qd + static_cast<uint32_t>(tile * C::kOp >> 4), bb = kd + static_cast<uint32_t>((at & 1) * C::kOp >> 4);
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          const int off = ((d / 4) * 16384 + (d % 4) * 32) >> 4;
          tc_mma_ss(tmem + tile * 128, a + off, bb + off, qk, d > 0);
        }
        tc_commit(&c->sfull[tile]);
      };
      auto values = [&](int tile, int at, bool acc) {
        const uint64_t bb = vd + static_cast<uint32_t>((at & 1) * C::kOp >> 4);
#pragma unroll
        for (int j = 0; j < kBlk / 16; ++j)
          tc_mma_ts(tmem + 256 + tile * 128, tmem + tile * 128 + j * 8, bb + (j * 2048 >> 4), wv, acc || j > 0);
      };
      bool live = true;
      int kb = 0, nb[2] = {0, 0}, ni[2] = {0, 0};  // blocks in all; of each tile; items of each tile
      for (int item = blockIdx.x; item < items && live; item += gridDim.x) {
        const TileItem I(P, item, blocks);
        if (I.nblk == 0) continue;
        for (int t = 0; t < I.tiles && live; ++t) {
          live = wait_on(c, &c->qfull[t], ni[t] & 1, limit);
          if (live && t == 0) live = wait_on(c, &c->kfull[kb & 1], (kb >> 1) & 1, limit);
          if (!live) break;
          tc_fence_after();
          scores(t, kb);
        }
        if (live) tc_commit(&c->kfree[kb & 1]);
        for (int k = 0; k < I.nblk && live; ++k) {
          const int at = kb + k;
          for (int t = 0; t < I.tiles && live; ++t) {
            live = wait_on(c, &c->pfull[t], (nb[t] + k) & 1, limit);
            if (live && t == 0) live = wait_on(c, &c->vfull[at & 1], (at >> 1) & 1, limit);
            // the item before's answers have to be out of the sums
            if (live && k == 0 && ni[t] > 0) live = wait_on(c, &c->ofree[t], (ni[t] - 1) & 1, limit);
            if (!live) break;
            tc_fence_after();
            values(t, at, k > 0);
            if (k + 1 < I.nblk) {
              if (t == 0) live = wait_on(c, &c->kfull[(at + 1) & 1], ((at + 1) >> 1) & 1, limit);
              if (!live) break;
              tc_fence_after();
              scores(t, at + 1);
            } else {
              tc_commit(&c->done[t]);
            }
          }
          if (live) {
            tc_commit(&c->vfree[at & 1]);
            if (k + 1 < I.nblk) tc_commit(&c->kfree[(at + 1) & 1]);
          }
        }
        kb += I.nblk;
        for (int t = 0; t < I.tiles; ++t) nb[t] += I.nblk, ++ni[t];
      }
      if (!live) {  // let what was issued end before tensor memory is given back
        tc_commit(&c->drain);
        mbar_wait_bounded(&c->drain, 0, limit);
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmax));
    const int tile = role, rr = tid;  // tile and row of the block: tile * 128 + lane of tensor memory
    const int wt = tid % 128;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t s_addr = lane_addr + tile * 128, o_addr = lane_addr + 256 + tile * 128;
    const float sc = fmaxf(fabsf(P.scale), 1e-37f);  // not zero: a key that is not seen has the score -inf
    bool live = true;
    int nb = 0, ni = 0, odd_at = 0;
    if (tree) grid_dependency_wait();

    // Queries of the tile's rows into shared memory: DP / 8 lanes per row, 16 bytes
    // each.  A negative scale turns their sign.
    auto load_queries = [&](const TileItem &I) {
      const int r = I.r0 + rr;
      long long off = -1;
      if (r < P.N * P.G) {
        const int t = r / P.G, h = I.g * P.G + (r - t * P.G);
        off = I.b * P.qs[0] + t * P.qs[1] + h * P.qs[2];
      }
      c->qoff[rr][0] = static_cast<int>(off);
      c->qoff[rr][1] = static_cast<int>(off >> 32);
      if (tile == 0)
        asm volatile("bar.sync 2, 128;" ::: "memory");
      else
        asm volatile("bar.sync 3, 128;" ::: "memory");
      constexpr int L = DP / 8, kBatch = L, kStep = 128 / L;
      const bool vec = reinterpret_cast<uintptr_t>(P.q) % 16 == 0 && P.qs[0] % 8 == 0 && P.qs[1] % 8 == 0 && P.qs[2] % 8 == 0;
      const int pc = wt % L, rr0 = wt / L;
      uint4 u[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = tile * 128 + rr0 + i * kStep;
        const long long o = static_cast<long long>(static_cast<uint32_t>(c->qoff[row][0])) | static_cast<long long>(c->qoff[row][1]) << 32;
        u[i] = make_uint4(0, 0, 0, 0);
        if (o >= 0 && pc * 8 < P.D) {
          const unsigned short *q = static_cast<const unsigned short *>(P.q) + o + pc * 8;
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
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = rr0 + i * kStep;
        if (P.scale < 0.f) u[i].x ^= 0x80008000u, u[i].y ^= 0x80008000u, u[i].z ^= 0x80008000u, u[i].w ^= 0x80008000u;
        *reinterpret_cast<uint4 *>(smem + C::kQ + tile * C::kOp + (pc / 8) * 16384 + row * 128 + (((pc % 8) ^ (row & 7)) << 4)) = u[i];
      }
      fence_async_smem();
      mbar_arrive(&c->qfull[tile]);
    };
    // the tile's next item with work, from `item` on
    auto next_item = [&](int item) {
      for (; item < items; item += gridDim.x) {
        const TileItem I(P, item, blocks);
        if (I.nblk > 0 && tile < I.tiles) break;
      }
      return item;
    };
    {
      const int item = next_item(blockIdx.x);
      if (item < items) load_queries(TileItem(P, item, blocks));
    }
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      const TileItem I(P, item, blocks);
      if (tile >= I.tiles) {
        if (I.nblk > 0) ++odd_at;
        continue;
      }
      const int r = I.r0 + rr;
      int at = -1, my = 0;  // the thread's output row (-1: past the last) and token
      if (r < P.N * P.G) {
        my = r / P.G;
        at = (I.b * P.N + my) * P.Hq + I.g * P.G + (r - my * P.G);
      }
      const bool use = at >= 0 && my < I.cnt;
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
      if (I.nblk == 0) {
        if (wt == 0 && tile == 0 && P.splits > 1) P.oflag[flag] = 0;
        empty(false);
        continue;
      }
      const bool mine = use && (!tree || P.rowinfo[I.b] >= 0);
      const int p = I.n + (tree ? mine ? P.depth[static_cast<size_t>(I.b) * P.N + my] : 0 : my);
      const int from = window_from(P, p);
      const uint32_t *const anc = tree ? P.anc + (static_cast<size_t>(I.b) * P.N + my) * P.W : nullptr;
      const Keys keys(P, I.p0, I.end);
      // the tile's own positions
      const int q_first = (I.r0 + tile * 128) / P.G, q_last = min((I.r0 + tile * 128 + 127) / P.G, P.N - 1);
      const int p0 = tree ? I.p0 : I.n + q_first, p1 = tree ? I.p1 : I.n + q_last;
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < I.nblk; ++k) {
        if (live) live = wait_on(c, &c->sfull[tile], (nb + k) & 1, limit);
        live = __all_sync(FULL_MASK, live);
        if (!live) break;
        tc_fence_after();
        unsigned part = 0;  // groups of the block that some query of the tile does not see whole
        {
          const int gi = I.g0 + k * kBlkGroups + (lane & 7);
          part = __ballot_sync(FULL_MASK, gi >= I.g1 || group_masked(P, keys.token(gi), I.n, p0, p1)) & 0xffu;
        }
        auto hide = [&](uint32_t (&x)[32], int q) {  // columns 32 q on: groups 2 q and 2 q + 1
          if (part >> (2 * q) & 3u) {
            const int gi = I.g0 + k * kBlkGroups + 2 * q;
            const uint32_t lo = gi < I.g1 ? group_seen(P, keys.token(gi), p, from, I.n, I.end, anc) : 0u;
            const uint32_t hi = gi + 1 < I.g1 ? group_seen(P, keys.token(gi + 1), p, from, I.n, I.end, anc) : 0u;
            const uint32_t bits = lo | hi << 16;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits >> j & 1)) x[j] = 0xff800000u;
          }
        };
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
        hide(s[0], 2);
        hide(s[1], 3);
        mq[2] = largest(s[0]);
        mq[3] = largest(s[1]);
        tc_ld32(s[0], s_addr);
        tc_ld32(s[1], s_addr + 32);
        tc_wait_ld();
        hide(s[0], 0);
        hide(s[1], 1);
        mq[0] = largest(s[0]);
        mq[1] = largest(s[1]);
        const float mt = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sc;
        float al = 1.f;
        if (mt > m + kTileLazy || m == -INFINITY) {
          al = mt == -INFINITY ? 1.f : ex2(m - mt);
          m = mt;
        }
        if (k > 0 && __any_sync(FULL_MASK, al != 1.f)) {
#pragma unroll
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
        tc_wait_ld();
        tc_ld32(s[1], s_addr + 96);
        hide(s[0], 2);
        weights(s[0], 2);
        tc_wait_ld();
        hide(s[1], 3);
        weights(s[1], 3);
        l = fmaf(l, al, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c->pfull[tile]);
      }
      nb += I.nblk;
      // the next queries may come: this item's scores are all taken
      if (live) {
        const int next = next_item(item + gridDim.x);
        if (next < items) load_queries(TileItem(P, next, blocks));
      }
      if (live) live = wait_on(c, &c->done[tile], ni & 1, limit);
      live = __all_sync(FULL_MASK, live);
      ++ni;
      grid_dependency_wait();  // the row's check
      if (!live) {
        empty(true);
        if (wt == 0 && tile == 0 && P.splits > 1) P.oflag[flag] = 0;
        ++odd_at;
        continue;
      }
      tc_fence_after();
      const bool odd = *reinterpret_cast<volatile int *>(&c->odd[odd_at & 3]) == item + 1;
      const bool some = use && P.rowinfo[I.b] >= 0 && l != 0.f;
      const float z = some ? m + log2f(l) : -INFINITY;
      if (P.splits > 1) {
        if (wt == 0 && tile == 0) P.oflag[flag] = odd;
        if (at >= 0) P.ml[ml_at] = some ? make_float2(m, z) : make_float2(-INFINITY, -INFINITY);
        float *const to = P.part + ml_at * P.D;
#pragma unroll
        for (int q = 0; q < DP / 32; ++q) {
          uint32_t o[32];
          __syncwarp();
          tc_ld32(o, o_addr + q * 32);
          tc_wait_ld();
          if (some) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (q * 32 + j < P.D) st_global_v8(to + q * 32 + j, o + j);
          }
        }
      } else {
        const float w = some ? ex2(m - z) : 0.f;
        if (at >= 0 && P.lse) P.lse[at] = kLn2 * z;
#pragma unroll
        for (int q = 0; q < DP / 32; ++q) {
          uint32_t o[32];
          __syncwarp();
          tc_ld32(o, o_addr + q * 32);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = some ? __float_as_uint(__uint_as_float(o[j]) * w) : 0u;
          if (some && odd)
            for (int j = 0; j < 32 && q * 32 + j < P.D; ++j) {
              const float y = paged_odd_sum<CT>(P, I.b, my, I.cnt, I.n, p, I.g, q * 32 + j);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e == j) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
            }
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            if (at >= 0 && q * 32 + j < P.D) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = pack16<BF>(__uint_as_float(o[j + 2 * e]), __uint_as_float(o[j + 2 * e + 1]));
              *reinterpret_cast<uint4 *>(answer + q * 32 + j) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
      }
      tc_fence_before();
      mbar_arrive(&c->ofree[tile]);
      ++odd_at;
    }
  }
  __syncthreads();
  grid_dependency_wait();
  if (warp == kIssueWarp) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem);
  }
}

template <int CT, int DP>
cudaError_t launch(const PagedParams &p, cudaStream_t s) {
  using C = Layout<DP>;
  const int blocks = (p.N * p.G + 255) / 256;
  const long long items = static_cast<long long>(p.B) * p.H * blocks * p.splits;
  if (items > 0x7fffffffLL - 4096) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<paged_tile_kernel<CT, DP>>(C::kSmem, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(items < kPagedSms ? items : kPagedSms);
  return launch_after(paged_tile_kernel<CT, DP>, dim3(grid), kTileThreads, C::kSmem, s, true, p, blocks, static_cast<int>(items));
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
