// prefix_attention_tile.cu -- spec_prefix_attention for many query rows:
// two tiles of 128 query rows of one KV head against a range of tokens, on
// the 5th-generation tensor cores.
//
// For 256 rows the two products cost 4 * 256 * D operations per token and head,
// about as long on the tensor cores as the softmax's exponentials between
// them, while the cache's bytes come mostly from L2 (every block of 256 rows
// reads the same prefix).  So the kernel is laid out to keep the tensor cores
// fed while the softmax runs:
//   - a CTA holds two row tiles A and B.  One thread issues, for each block of
//     128 tokens, W V and then the next Q K^T of tile A, then those of tile B;
//     while the tensor cores work on one tile, a warpgroup does the other's
//     softmax;
//   - scores, weights and sums stay in tensor memory (scores of A and B at
//     columns 0 and 128, sums at 256 and 384); the weights take the place of
//     the scores and are the product's left operand from there;
//   - a thread owns a row, so its softmax needs no exchange.  The sums are
//     rescaled only when a row's maximum has grown by more than 2^8 since
//     the last time (codes: before a weight would leave fp16's range): weights
//     up to 2^8 are as exact as weights up to 1;
//   - four warps bring keys and values into shared memory, two buffers each:
//     16-bit entries by asynchronous copies, e4m3 codes through registers as
//     fp16 numbers relative to the block's largest scale (exact for scales
//     down to 2^-15 of it), so that the block's scale is one factor on the
//     scores and one on the sums.  A part with a block whose scales lie further
//     apart is taken once more in fp32 (exact_part).
// Measured with 32 query heads and 8 KV heads of 128: a block of 128 tokens takes
// both tiles 1.84 us in bf16 (the products alone 1.6; 1.35 at the library's dense
// rate), an item's start and end about 11; 64 chains of 6 tokens behind 8192: 50
// us.  32 trees of 60 nodes in e4m3: 202 us, two rounds of items where 1.7 would
// do.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.cuh"
#include "internal.h"

namespace sv {
namespace {

constexpr int kTok = 128;          // tokens per block, a producer thread each
// Groups of 128 threads: softmax of tiles A and B, producers, tensor-core
// issue.  Their registers per thread add up to what the block is launched
// with, and are split so that the loops hold what they need (12 to 20 bytes spill
// in three of the variants for codes): with 160 for the softmax
// and 120 for producers of codes, 32 trees of 60 nodes behind 4097 tokens take
// 212 us where this split takes 201.  (Two groups of producers, 96 registers a
// thread, were 8 % slower than one.)
template <bool E4>
struct Roles {
  static constexpr int kGroups = 4, kThreads = 128 * kGroups, kProducers = 128;
  static constexpr int kIssueWarp = 4 * (kGroups - 1);
  static constexpr int kLaunch = 128;  // registers per thread at launch: 65536 / kThreads
  static constexpr int kSoftmax = E4 ? 176 : 184, kProduce = E4 ? 88 : 72, kIssue = 72;
  static_assert(kSoftmax > kLaunch && kProduce < kLaunch && kIssue < kLaunch, "softmax takes more, the others give back");
  static_assert(2 * kSoftmax + kProduce + kIssue == kGroups * kLaunch, "the block's registers");
};
constexpr float kLazy = 8.f;       // 16-bit caches: log2 of the growth a row's maximum may make before its sums follow

template <int DP>
struct TileCfg {
  static constexpr int kOp = kTok * DP * 2;  // an operand tile: 128 rows, 64-column panels of 16 KB
  static constexpr int kQ = 0;               // tiles A and B
  static constexpr int kK = 2 * kOp;         // two buffers
  static constexpr int kV = 4 * kOp;         // two buffers
  static constexpr int kCtrl = 6 * kOp;
  static constexpr int kSmem = kCtrl + 7168 + 1024;  // + control block + alignment
};

struct Ctrl {
  uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  uint64_t sfull[2], pfull[2], done[2], qfull, drain;
  uint32_t tmem;
  int abort;
  int odd;
  int far_apart;            // scales that the conversion or the sums do not span: exact_part
  float ksc[2];             // per buffer: the block's scale of the keys
  float vex[2], vtop[2];    // the values' exponent, and the largest so far
  int uneven[2];            // the values' scales differ by more than kEvenSpan
  uint32_t red[2][4];       // producers' reductions
  uint32_t mult[2][128];    // fp16 factors of the block's tokens, keys and values
  float qfac[256];
  long long qoff[256];      // where a query row's elements are; -1: past the last
};
static_assert(sizeof(Ctrl) <= 7168, "control block");
// l counts in units of 2^(m - E): with exponents no further apart than this it
// stays in fp32's range for any number of tokens
constexpr float kSumSpan = 80.f;
// Codes: a row's reference m must not pass max_t (x_t + e_t) over the tokens it
// sees, or weights that count are lost in fp16's steps.  What is at hand of a block
// is its largest score and its largest exponent, ex, which may be different
// tokens' (one that nothing sees, one whose weight is nothing).  So m is put
// below their sum: by kEvenBelow where all exponents lie within kEvenSpan of ex,
// else by kUnevenBelow, as far as exponents can lie below ex (further down, only
// zeros: a vector of zeros with more than 2^15 times all other weight is the one
// thing that still costs the others bits, on a grid of 2^-39 of the whole).  m
// follows only before a weight would leave fp16's range, 2^kWeightTop.
constexpr float kEvenSpan = 4.f, kEvenBelow = 4.5f, kUnevenBelow = 15.f, kWeightTop = 15.5f;
constexpr float kUnevenMark = 1024.f;  // added to a converted block's value exponent
constexpr int kUnused = 1 << 30;  // the row has no such query (its answer is empty)

// ------------------------------------------------------------ tcgen05 wrappers
__device__ __forceinline__ void tc_alloc(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (tensor memory) = A (shared) B (shared) [+ D]
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// D (tensor memory) = A (tensor memory) B (shared) [+ D]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// 32 columns of this thread's lane
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle: rows of 128 bytes in
// groups of 8 (1024 bytes).  A tile of rows x 64 columns is one panel; for an
// operand whose 64-column direction is the product's M or N (the values), the
// leading offset is the distance of two panels.
__device__ __forceinline__ uint64_t op_desc(uint32_t addr, uint32_t panel) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>(panel >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: fp32 sums, 16-bit operands, M = 128.
__device__ __forceinline__ uint32_t inst_desc(bool bf16, int n, bool b_cols) {
  const uint32_t f = bf16 ? 1u : 0u;
  return 1u << 4 | f << 7 | f << 10 | (b_cols ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void producer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// Bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool wait_for(Ctrl *c, uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
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

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Items.  PRE: the prefix alone, for (KV head, block of 256 rows of all rows'
// queries, part).  Else (row, KV head, block of 256 of the row's queries,
// part) against the row's own entries, after the prefix's if P.fuse; with one
// part and nothing else to join (P.direct) it writes the answer itself.
template <int CT, int DP, bool PRE>
__global__ void __launch_bounds__(Roles<CT == SPEC_E4M3>::kThreads, 1) attn_tile_kernel(const __grid_constant__ AttnParams P, int blocks) {
  using C = TileCfg<DP>;
  using R = Roles<CT == SPEC_E4M3>;
  constexpr int kProducers = R::kProducers;
  constexpr bool E4 = CT == SPEC_E4M3, BF = CT == SPEC_BF16;
  extern __shared__ unsigned char raw[];
  unsigned char *const smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctrl *const c = reinterpret_cast<Ctrl *>(smem + C::kCtrl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, role = tid / 128;

  grid_dependency_wait();

  // --- the item
  int item = blockIdx.x;
  const int nsplit = PRE ? P.psplits : P.osplits;
  const int split = item % nsplit;
  item /= nsplit;
  const int blk = item % blocks;
  item /= blocks;
  const int g = PRE ? item : item % P.H;
  const int b = PRE ? 0 : item / P.H;
  const int r0 = blk * 256;
  const int nrows = (PRE ? P.B : 1) * P.N * P.G;
  const int slot = PRE ? split : P.psplits + split;
  // blocks of tokens: the prefix's npre first, then the row's own; this part
  // takes n of them from block q0 on
  int npre = PRE || P.fuse ? (P.P + kTok - 1) / kTok : 0;
  int q0, n, len0 = 0, len = 0, cnt = 0;
  if constexpr (PRE) {
    q0 = split * (P.pchunk / kTok);
    n = min(P.pchunk / kTok, npre - q0);
  } else {
    cnt = row_queries(P, b);
    len0 = __ldg(P.kv_len + b);
    len = len0 + cnt;
    if (split == 0 && blk == 0 && g == 0 && tid == 0 && P.row_status && !P.direct)  // P.direct: the mask kernel has
      P.row_status[b] = cnt >= 0 ? 0 : cnt == kRowBadParent ? SPEC_ROW_BAD_PARENT : SPEC_ROW_BAD_SLOT;
    const int all = cnt > 0 ? npre + (len + kTok - 1) / kTok : 0, per = (all + nsplit - 1) / nsplit;
    q0 = split * per;
    n = max(0, min(per, all - q0));
  }
  const int tiles = nrows - r0 > 128 ? 2 : 1;       // row tiles in use
  if (n == 0) {  // nothing here (an empty part, or a row that cannot be used)
    if (tid < 256 && r0 + tid < nrows) {
      const int t = (r0 + tid) / P.G;
      const long long at = static_cast<long long>((PRE ? 0 : b) * P.N + t) * P.Hq + g * P.G + (r0 + tid - t * P.G);
      if (P.direct) {
        for (int d = 0; d < P.D; d += 8) *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(P.out) + at * P.D + d) = make_uint4(0, 0, 0, 0);
        if (P.lse) P.lse[at] = -INFINITY;
      } else {
        P.ml[static_cast<long long>(slot) * P.rows + at] = make_float2(-INFINITY, -INFINITY);
      }
    }
    if (!PRE && tid == 0) P.oflag[blockIdx.x] = 0;
    return;
  }

  // --- set up: barriers and tensor memory
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->kfull[i], kProducers);
      mbar_init(&c->vfull[i], kProducers);
      mbar_init(&c->kfree[i], 1);
      mbar_init(&c->vfree[i], 1);
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->pfull[i], 128);
      mbar_init(&c->done[i], 1);
    }
    mbar_init(&c->qfull, 256);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    c->odd = 0;
    c->far_apart = 0;
    fence_mbar_init();
  }
  if (warp == R::kIssueWarp) tc_alloc(&c->tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const uint64_t limit = P.wait_limit_ns;

  if (role >= 2 && role < R::kGroups - 1) {
    // ------------------------------------------------------------ producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kProduce));
    const int pt = tid - 256;
    bool live = true;
    // A thread brings 16-byte pieces of every kStep-th token.  Item 2k: keys
    // of block k, item 2k + 1: its values.  16-bit entries go where the tensor
    // cores want them; codes land in the same buffer as they are and are turned
    // into fp16 there once they have arrived.
    constexpr int L = E4 ? DP / 16 : DP / 8, kStep = kProducers / L, kPer = kTok / kStep;
    const int pc = pt % L, row0 = pt / L;
    const bool col = pc * 16 < P.D * (E4 ? 1 : 2);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t put0 = E4 ? pt * 16 : (pc / 8) * 16384 + row0 * 128 + (((pc % 8) ^ (row0 & 7)) << 4);
    constexpr int kPut = E4 ? kProducers * 16 : kStep * 128;
    const long long src0 = static_cast<long long>(g) * P.D * (E4 ? 1 : 2) + (col ? pc * 16 : 0);
    const unsigned char *const ok = P.k + b * P.row_stride, *const ov = P.v + b * P.row_stride;
    // copies of item it; for codes, the scale byte of the block's token pt (of a
    // prefix that is fp16 already, the bits of the block's scale)
    auto issue = [&](int it) -> uint32_t {
      uint32_t byte = 0;
      if (it < 2 * n) {
        const int k = it >> 1, s = k & 1, q = q0 + k;
        const bool pre = PRE || q < npre, val = it & 1;
        const int tb = (pre ? q : q - npre) * kTok, left = (pre ? P.P : len) - tb;
        if constexpr (E4) {
          if (pre && P.wide) {
            constexpr int WL = DP / 8, kWStep = kProducers / WL;
            const int wc = pt % WL, wrow = pt / WL;
            const long long ts = static_cast<long long>(P.H) * P.D * 2;
            const unsigned char *src = P.wide + (static_cast<long long>(val ? P.P : 0) + tb + wrow) * ts + static_cast<long long>(g) * P.D * 2 + wc * 16;
            byte = __float_as_uint(__ldg(P.wide_scale + (static_cast<long long>(val ? P.H : 0) + g) * npre + q));
            if (k >= 2 && live) live = wait_for(c, val ? &c->vfree[s] : &c->kfree[s], ((k >> 1) - 1) & 1, limit);
            if (live) {
              const uint32_t dst = sbase + (val ? C::kV : C::kK) + s * C::kOp + (wc / 8) * 16384 + wrow * 128 + (((wc % 8) ^ (wrow & 7)) << 4);
              const bool in = wc * 16 < P.D * 2;
#pragma unroll
              for (int i = 0; i < kTok / kWStep; ++i) {
                const bool on = in && wrow + i * kWStep < left;
                cp_async16_zfill(dst + i * kWStep * 128, on ? src : P.wide, on);
                src += ts * kWStep;
              }
            }
            cp_async_commit();
            return byte;
          }
        }
        const long long ts = pre ? P.ptok_stride : P.tok_stride;
        const unsigned char *const base = (pre ? (val ? P.pv : P.pk) : (val ? ov : ok)) + tb * ts;
        if constexpr (E4)
          if (pt < left) byte = __ldg(base + pt * ts + static_cast<long long>(P.H) * P.D + g);
        if (k >= 2 && live) live = wait_for(c, val ? &c->vfree[s] : &c->kfree[s], ((k >> 1) - 1) & 1, limit);
        if (live) {
          const unsigned char *src = base + src0 + row0 * ts;
          const uint32_t dst = sbase + put0 + (val ? C::kV : C::kK) + s * C::kOp;
          const long long step = ts * kStep;
          if (col && row0 + (kPer - 1) * kStep < left) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              cp_async16_zfill(dst + i * kPut, src, true);
              src += step;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const bool on = col && row0 + i * kStep < left;
              cp_async16_zfill(dst + i * kPut, on ? src : base, on);
              src += step;
            }
          }
        }
      }
      cp_async_commit();
      return byte;
    };
    float E = kMinExponent, low = 0.f, kscale = 1.f;  // the largest and smallest exponent of a block of values
    uint32_t sc0 = issue(0), sc1 = issue(1);
    for (int it = 0; it < 2 * n; ++it) {
      cp_async_wait<1>();
      const int k = it >> 1, s = k & 1, q = q0 + k;
      const bool val = it & 1;
      // From this row of the block on, values are the pass's own tokens'.
      // Those that are not finite are taken out (a query that does not see
      // them would get 0 * NaN) and put into the answers of the queries that
      // see them at the end.
      const int own0 = !PRE && val && q >= npre ? len0 - (q - npre) * kTok : kTok;
      if constexpr (!E4) {
        if (own0 < kTok && live) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (row0 + i * kStep < own0) continue;
            const uint32_t at = sbase + put0 + C::kV + s * C::kOp + i * kPut;
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              constexpr uint32_t top = BF ? 0x7f80u : 0x7c00u;
              if ((w[e] & top) == top) w[e] &= 0xffff0000u, odd = true;
              if ((w[e] >> 16 & top) == top) w[e] &= 0x0000ffffu, odd = true;
            }
            if (odd) {
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
              c->odd = 1;
            }
          }
        }
      } else if ((PRE || q < npre) && P.wide) {
        if (!val) kscale = __uint_as_float(sc0);
        if (pt == 0 && __ldg(P.wide_far + (static_cast<long long>(val ? P.H : 0) + g) * npre + q)) c->far_apart = 1;
        if (val) {
          float ex = __uint_as_float(sc0);
          if (ex > kUnevenMark / 2) ex -= kUnevenMark;
          E = fmaxf(E, ex);
          low = fminf(low, ex);
          if (pt == 0) {
            if (E - low > kSumSpan) c->far_apart = 1;
            c->ksc[s] = kscale;
            c->vex[s] = ex;
            c->vtop[s] = E;
          }
        }
      } else {
        const uint32_t buf = sbase + (val ? C::kV : C::kK) + s * C::kOp;
        uint32_t w[kPer][4];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                       : "r"(buf + put0 + i * kPut)
                       : "memory");
        // the block's largest scale
        const uint32_t wtop = __reduce_max_sync(FULL_MASK, sc0 == 255u ? 1u : max(sc0, 1u));
        if (lane == 0) c->red[it & 1][pt / 32] = wtop;
        if (val && pt == 0) c->uneven[s] = 0;
        producer_sync<kProducers>();  // also: every code of the block has been read
        const uint32_t top = max(max(c->red[it & 1][0], c->red[it & 1][1]), max(c->red[it & 1][2], c->red[it & 1][3]));
        float ex = static_cast<float>(static_cast<int>(top) - 127);
        if (val) {
          E = fmaxf(E, ex);
          ex = fmaxf(ex, E - kExponentSpan);
          low = fminf(low, ex);
          if (pt == 0 && E - low > kSumSpan) c->far_apart = 1;
        }
        {
          // 2^(scale - block's scale) as fp16: exact down to 2^-24, zero below
          const int d = static_cast<int>(sc0) - (static_cast<int>(ex) + 127);
          const uint32_t f = sc0 == 255u ? 0x7e00u : d >= -14 ? static_cast<uint32_t>(d + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u;
          c->mult[it & 1][pt] = f | f << 16;
          if (d < -15 && sc0 > kLeastScale && sc0 != 255u) c->far_apart = 1;
          if (val && static_cast<float>(d) < -kEvenSpan && pt < (PRE || q < npre ? P.P - q * kTok : len - (q - npre) * kTok)) c->uneven[s] = 1;
        }
        producer_sync<kProducers>();
        const uint32_t dst = buf + (pc / 4) * 16384 + row0 * 128;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int row = row0 + i * kStep;
          const uint32_t fw = c->mult[it & 1][row];
          const __half2 f2 = *reinterpret_cast<const __half2 *>(&fw);
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = e4m3x2_to_f16x2(w[i][e]), hi = e4m3x2_to_f16x2_hi(w[i][e]);
            const __half2 l2 = __hmul2(*reinterpret_cast<const __half2 *>(&lo), f2);
            const __half2 h2 = __hmul2(*reinterpret_cast<const __half2 *>(&hi), f2);
            o[2 * e] = *reinterpret_cast<const uint32_t *>(&l2);
            o[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&h2);
          }
          if (row >= own0) {
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if ((o[e] & 0x7c00u) == 0x7c00u) o[e] &= 0xffff0000u, odd = true;
              if ((o[e] >> 16 & 0x7c00u) == 0x7c00u) o[e] &= 0x0000ffffu, odd = true;
            }
            if (odd) c->odd = 1;
          }
          // the two 16-byte halves, the upper panel's lanes in the other
          // order: eight lanes then cover all banks
          const int ch = (pc % 4) * 2, up = pc / 4;
          const uint32_t at = dst + i * kStep * 128;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((ch + up) ^ (row & 7)) << 4)),
                       "r"(up ? o[4] : o[0]), "r"(up ? o[5] : o[1]), "r"(up ? o[6] : o[2]), "r"(up ? o[7] : o[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((ch + 1 - up) ^ (row & 7)) << 4)),
                       "r"(up ? o[0] : o[4]), "r"(up ? o[1] : o[5]), "r"(up ? o[2] : o[6]), "r"(up ? o[3] : o[7])
                       : "memory");
        }
        // the keys' scale goes with the values' exponents: the softmax waits
        // for the values' buffer, which it holds until it is done
        if (!val) kscale = e4m3_scale(top);
        if (val && pt == 0) {
          c->ksc[s] = kscale;
          c->vex[s] = ex;
          c->vtop[s] = E;
        }
      }
      fence_async_smem();
      if (!(it == 0 && (P.force_timeout == 1 || P.force_timeout == g + 2))) mbar_arrive(val ? &c->vfull[s] : &c->kfull[s]);
      sc0 = sc1;
      sc1 = issue(it + 2);  // after this item is handed over: its buffer may be a while in coming free
    }
    cp_async_wait_all();
  } else if (role == R::kGroups - 1) {
    // ------------------------------------------------- tensor-core issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kIssue));
    if (warp == R::kIssueWarp && lane == 0) {
      const uint32_t qk = inst_desc(BF, kTok, false), wv = inst_desc(BF, DP, true);
      const uint32_t base = smem_u32(smem);
      const uint64_t qd = op_desc(base + C::kQ, 16), kd = op_desc(base + C::kK, 16), vd = op_desc(base + C::kV, 16384);
      auto scores = [&](int tile, int k) {
        const uint64_t a = qd + static_cast<uint32_t>(tile * C::kOp >> 4), bb = kd + static_cast<uint32_t>((k & 1) * C::kOp >> 4);
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          const int off = ((d / 4) * 16384 + (d % 4) * 32) >> 4;
          tc_mma_ss(tmem + tile * 128, a + off, bb + off, qk, d > 0);
        }
        tc_commit(&c->sfull[tile]);
      };
      auto values = [&](int tile, int k) {
        const uint64_t bb = vd + static_cast<uint32_t>((k & 1) * C::kOp >> 4);
#pragma unroll
        for (int j = 0; j < kTok / 16; ++j)
          tc_mma_ts(tmem + 256 + tile * 128, tmem + tile * 128 + j * 8, bb + (j * 2048 >> 4), wv, k > 0 || j > 0);
      };
      bool live = wait_for(c, &c->qfull, 0, limit) && wait_for(c, &c->kfull[0], 0, limit);
      if (live) {
        tc_fence_after();
        for (int t = 0; t < tiles; ++t) scores(t, 0);
        tc_commit(&c->kfree[0]);
      }
      for (int k = 0; k < n && live; ++k) {
        for (int t = 0; t < tiles && live; ++t) {
          live = wait_for(c, &c->pfull[t], k & 1, limit);
          if (live && t == 0) live = wait_for(c, &c->vfull[k & 1], (k >> 1) & 1, limit);
          if (!live) break;
          tc_fence_after();
          values(t, k);
          if (k + 1 < n) {
            if (t == 0) live = wait_for(c, &c->kfull[(k + 1) & 1], ((k + 1) >> 1) & 1, limit);
            if (!live) break;
            tc_fence_after();
            scores(t, k + 1);
          } else {
            tc_commit(&c->done[t]);
          }
        }
        if (live) {
          tc_commit(&c->vfree[k & 1]);
          if (k + 1 < n) tc_commit(&c->kfree[(k + 1) & 1]);
        }
      }
      if (!live) {  // let what was issued end before tensor memory is given back
        tc_commit(&c->drain);
        mbar_wait_bounded(&c->drain, 0, limit);
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmax));
    // --- queries of rows tid (table) and of all 256 rows (operand): DP/8 lanes
    // per row, 16 bytes each; fp16 for an e4m3 cache: a row far outside fp16's
    // range is brought into it by a power of two.  A negative scale turns the
    // queries' sign.
    int at = -1;  // the thread's output row; -1: past the last, kUnused: no such query
    {
      const int r = r0 + tid;
      long long off = -1;
      if (r < nrows) {
        const int t = r / P.G, h = g * P.G + (r - t * P.G);
        const int qb = PRE ? t / P.N : b, qt = PRE ? t - qb * P.N : t;
        at = (qb * P.N + qt) * P.Hq + h;
        off = qb * P.qs[0] + qt * P.qs[1] + h * P.qs[2];
      }
      c->qoff[tid] = off;
    }
    asm volatile("bar.sync 2, 256;" ::: "memory");
    {
      constexpr int L = DP / 8, kIt = L, kBatch = kIt, kStep = 256 / L;
      const bool vec = reinterpret_cast<uintptr_t>(P.q) % 16 == 0 && P.qs[0] % 8 == 0 && P.qs[1] % 8 == 0 && P.qs[2] % 8 == 0;
      const int pc = tid % L, rr0 = tid / L;
#pragma unroll
      for (int i0 = 0; i0 < kIt; i0 += kBatch) {
        uint4 u[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const long long off = c->qoff[rr0 + (i0 + i) * kStep];
          u[i] = make_uint4(0, 0, 0, 0);
          if (off >= 0 && pc * 8 < P.D) {
            const unsigned short *q = static_cast<const unsigned short *>(P.q) + off + pc * 8;
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
          const int rr = rr0 + (i0 + i) * kStep;
          float fac = 1.f;
          if (E4 && P.qbf16) {
            const float x[8] = {bf16_lo(u[i].x), bf16_hi(u[i].x), bf16_lo(u[i].y), bf16_hi(u[i].y),
                                bf16_lo(u[i].z), bf16_hi(u[i].z), bf16_lo(u[i].w), bf16_hi(u[i].w)};
            uint32_t a = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL_MASK, a, o));
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
          if (pc == 0) c->qfac[rr] = fac;
          if (P.scale < 0.f) u[i].x ^= 0x80008000u, u[i].y ^= 0x80008000u, u[i].z ^= 0x80008000u, u[i].w ^= 0x80008000u;
          *reinterpret_cast<uint4 *>(smem + C::kQ + (rr / 128) * C::kOp + (pc / 8) * 16384 + (rr % 128) * 128 + (((pc % 8) ^ (rr & 7)) << 4)) = u[i];
        }
      }
    }
    fence_async_smem();
    mbar_arrive(&c->qfull);
    // queries that a row does not have were read all the same: nothing of them is kept
    if (at >= 0) {
      const int t = (r0 + tid) / P.G, qb = PRE ? t / P.N : b;
      if ((PRE ? t - qb * P.N : t) >= (PRE ? row_queries(P, qb) : cnt)) at |= kUnused;
    }
    asm volatile("bar.sync 2, 256;" ::: "memory");  // the factors, for every row's thread
    const int tile = role;
    if (tile < tiles) {
      const int rr = tid;  // row of the block (tile * 128 + lane of tensor memory)
      const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp & 3) << 21);
      const uint32_t s_addr = lane_addr + tile * 128, o_addr = lane_addr + 256 + tile * 128;
      const float base_sc = fabsf(P.scale) * (E4 ? c->qfac[rr] : 1.f);
      const int my = PRE ? 0 : min((r0 + rr) / P.G, P.N - 1);  // the row's token
      const uint32_t *const anc = PRE || !P.anc ? nullptr : P.anc + (static_cast<size_t>(b) * P.N + my) * P.W;
      float m = -INFINITY, l = 0.f, E = E4 ? kMinExponent : 0.f;
      const float *const wscale = E4 && P.wide ? P.wide_scale + static_cast<long long>(g) * npre : nullptr;
      float kscale = 1.f, vexp = 0.f;
      if (E4 && P.wide && q0 < npre) {
        kscale = __ldg(wscale + q0);
        vexp = __ldg(wscale + static_cast<long long>(P.H) * npre + q0);
      }
      bool live = true;
      for (int k = 0; k < n; ++k) {
        live = wait_for(c, &c->sfull[tile], k & 1, limit);
        float ex = 0.f, sc = base_sc, grow = 0.f, below = 0.f;
        if constexpr (E4) {
          float En;
          if ((PRE || q0 + k < npre) && P.wide) {
            // a converted prefix's scales, read a block ahead: the softmax need not wait for the values
            sc *= kscale;
            ex = vexp;
            below = kEvenBelow;
            if (ex > kUnevenMark / 2) ex -= kUnevenMark, below = kUnevenBelow;
            En = fmaxf(E, ex);
            if (k + 1 < n && q0 + k + 1 < npre) {
              kscale = __ldg(wscale + q0 + k + 1);
              vexp = __ldg(wscale + static_cast<long long>(P.H) * npre + q0 + k + 1);
            }
          } else {
            if (live) live = wait_for(c, &c->vfull[k & 1], (k >> 1) & 1, limit);
            sc *= c->ksc[k & 1];
            ex = c->vex[k & 1];
            below = c->uneven[k & 1] ? kUnevenBelow : kEvenBelow;
            En = c->vtop[k & 1];
          }
          grow = En - E;
          E = En;
        }
        sc = fmaxf(sc, 1e-37f);  // not zero: a token that is not seen has the score -inf
        live = __all_sync(FULL_MASK, live);
        if (!live) break;
        tc_fence_after();
        const int q = q0 + k;
        const bool pre = PRE || q < npre;
        const int tb = (pre ? q : q - npre) * kTok;
        const bool masked = tb + kTok > (pre ? P.P : len0);
        // which of the 32 tokens from column 32 c32 this row sees
        auto seen = [&](int c32) -> uint32_t {
          const int tq = tb + c32 * 32;
          uint32_t bits;
          if (pre || !anc) {
            const int see = (pre ? P.P : min(len, len0 + my + 1)) - tq;
            bits = see >= 32 ? 0xffffffffu : see <= 0 ? 0u : (1u << see) - 1u;
          } else {
            const int j = tq - len0;  // first token's index among the pass's own
            if (j <= -32) {
              bits = 0xffffffffu;
            } else if (j < 0) {
              bits = ((1u << -j) - 1u) | __ldg(anc) << -j;
            } else {
              const int wd = j >> 5;
              const uint32_t lo = wd < P.W ? __ldg(anc + wd) : 0u, hi = wd + 1 < P.W ? __ldg(anc + wd + 1) : 0u;
              bits = __funnelshift_r(lo, hi, j & 31);
            }
            const int in = len - tq;
            if (in < 32) bits &= in <= 0 ? 0u : (1u << in) - 1u;
          }
          return bits;
        };
        // 64 of the row's 128 scores are held at a time (all of them do not fit
        // in registers beside the rest): the upper half is read for the maximum,
        // then the lower half, whose weights are taken first, then the upper
        // half again.
        uint32_t s[2][32];
        auto hide = [&](uint32_t (&x)[32], int q) {
          if (masked) {
            const uint32_t bits = seen(q);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits >> j & 1)) x[j] = 0xff800000u;
          }
        };
        auto largest = [](const uint32_t (&x)[32]) {
          float y = __uint_as_float(x[0]), z = __uint_as_float(x[1]);
#pragma unroll
          for (int j = 2; j < 30; j += 4) {
            y = max3(y, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
            z = max3(z, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
          }
          return fmaxf(max3(y, __uint_as_float(x[30]), __uint_as_float(x[31])), z);
        };
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
        const float top = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        const float mt = top == -INFINITY ? -INFINITY : fmaf(top, sc, ex);
        float al = 1.f;
        const float old = m;
        if (mt > m + (E4 ? kWeightTop : kLazy) || m == -INFINITY) {
          const float to = E4 ? mt - below : mt;
          al = to == -INFINITY ? 1.f : ex2(m - to);
          m = to;
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
        const float2 sc2 = make_float2(sc, sc), off2 = make_float2(ex - ref, ex - ref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weights = [&](const uint32_t (&x)[32], int q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = ffma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sc2, off2);
            const float2 p = make_float2(ex2(y.x), ex2(y.y));
            sum[j & 1] = fadd2(sum[j & 1], p);
            pk[j] = pack16<BF>(p.x, p.y);
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
        const float add = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if constexpr (E4) {
          // l counts in units of 2^(m - E)
          const float ll = grow != 0.f ? (old == -INFINITY ? 0.f : ex2(old - m + grow)) : al;
          l = fmaf(l, ll, add * ex2(fminf(E - ex, 126.f)));
        } else {
          l = fmaf(l, al, add);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c->pfull[tile]);
      }
      if (live) live = __all_sync(FULL_MASK, wait_for(c, &c->done[tile], 0, limit));
      if (PRE && P.next) allow_dependents();  // the rows kernel's items may take the SMs as they come free
      const long long orow = at & (kUnused - 1);
      float2 *const ml = P.ml + static_cast<long long>(slot) * P.rows + orow;
      if (!live) {
        if (at >= 0 && !P.direct) *ml = make_float2(-INFINITY, __uint_as_float(kTimeoutBits));
        if (at >= 0 && P.direct) {
          for (int d = 0; d < P.D; d += 8) *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(P.out) + orow * P.D + d) = make_uint4(0, 0, 0, 0);
          if (P.lse) P.lse[orow] = -INFINITY;
          if (P.row_status) P.row_status[b] = SPEC_ROW_TIMEOUT;
        }
      } else {
        tc_fence_after();
        const bool some = at >= 0 && at < kUnused && l != 0.f;
        const float z = some ? m + log2f(l) - E : -INFINITY;
        if (E4 && c->far_apart) {
          if (at >= 0)
            exact_part(P, b, g, q0 * kTok, min(min(q0 + n, npre) * kTok, P.P), max(0, q0 - npre) * kTok, min((q0 + n - npre) * kTok, len), len0, cnt,
                       my, anc, at < kUnused, c->qoff[rr], orow, slot, c->odd);
        } else if (P.direct) {  // every thread loads: tensor memory is read by whole warps
          const float w = some ? ex2(m - z) : 0.f;
          const bool odd = some && c->odd;
          if (at >= 0 && P.lse) P.lse[orow] = kLn2 * z;
#pragma unroll
          for (int q = 0; q < DP / 32; ++q) {
            uint32_t o[32];
            __syncwarp();
            tc_ld32(o, o_addr + q * 32);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = some ? __float_as_uint(__uint_as_float(o[j]) * w) : 0u;
            if (odd)  // values that are not finite, of the pass's tokens that this query sees
              for (int t = 0; t < cnt; ++t)
                if (anc ? anc[t >> 5] >> (t & 31) & 1u : t <= my)
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (q * 32 + j < P.D) o[j] = __float_as_uint(__uint_as_float(o[j]) + odd_value<CT>(P, b, len0 + t, g, q * 32 + j));
            unsigned short *const to = static_cast<unsigned short *>(P.out) + orow * P.D + q * 32;
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (at >= 0 && q * 32 + j < P.D) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float lo = __uint_as_float(o[j + 2 * e]), hi = __uint_as_float(o[j + 2 * e + 1]);
                  y[e] = P.qbf16 ? pack16<true>(lo, hi) : pack16<false>(lo, hi);
                }
                *reinterpret_cast<uint4 *>(to + j) = make_uint4(y[0], y[1], y[2], y[3]);
              }
          }
        } else {
          if (at >= 0) *ml = some ? make_float2(m, z) : make_float2(-INFINITY, -INFINITY);
          float *const to = P.part + (static_cast<long long>(slot) * P.rows + orow) * P.D;
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
        }
        tc_fence_before();
      }
    }
  }
  __syncthreads();
  if (!PRE && tid == 0) P.oflag[blockIdx.x] = c->odd;
  if (warp == R::kIssueWarp) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem);
  }
}

// ------------------------------------------------------ a prefix read often
// An e4m3 prefix that many blocks of query rows will read is turned into fp16
// once: 128 tokens of a head and plane per CTA, relative to their largest scale
// as the tile kernel does it.  Costs one read of the codes and one write of
// twice as many bytes, and saves every item the conversion, which takes longer
// than the tensor cores do (a block of tokens: 3.2 us with it, 1.8 without).
constexpr int kWidenThreads = 256;
__global__ void __launch_bounds__(kWidenThreads) attn_widen_kernel(const __grid_constant__ AttnParams P) {
  __shared__ uint32_t warp_top[4];
  __shared__ uint32_t mult[kTok];
  const int blk = blockIdx.x, g = blockIdx.y, val = blockIdx.z, tid = threadIdx.x;
  allow_dependents();
  const int tb = blk * kTok, left = P.P - tb;
  const unsigned char *const base = (val ? P.pv : P.pk) + tb * P.ptok_stride;
  uint32_t byte = 0;
  int far = 0, uneven = 0;
  if (tid < kTok) {
    if (tid < left) byte = __ldg(base + tid * P.ptok_stride + static_cast<long long>(P.H) * P.D + g);
    const uint32_t top = __reduce_max_sync(FULL_MASK, byte == 255u ? 1u : max(byte, 1u));
    if (tid % 32 == 0) warp_top[tid / 32] = top;
  }
  // two 16-code pieces of tokens a thread, while the scales settle
  const int parts = P.D / 16, pieces = kTok * parts;
  constexpr int kMost = kTok * (SPEC_MAX_HEAD_DIM / 16) / kWidenThreads;
  uint4 w[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int x = i * kWidenThreads + tid, t = x / parts, pc = x - t * parts;
    if (x < pieces && t < left) w[i] = __ldg(reinterpret_cast<const uint4 *>(base + t * P.ptok_stride + static_cast<long long>(g) * P.D + pc * 16));
  }
  __syncthreads();
  // scales below 2^-120 count as that: nothing they hold is seen beside the least exponent of the sums
  const int ref = max(static_cast<int>(kLeastScale), static_cast<int>(max(max(warp_top[0], warp_top[1]), max(warp_top[2], warp_top[3]))));
  if (tid < kTok) {
    const int d = static_cast<int>(byte) - ref;
    const uint32_t f = byte == 255u ? 0x7e00u : d >= -14 ? static_cast<uint32_t>(d + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u;
    mult[tid] = f | f << 16;
    far = d < -15 && byte > kLeastScale && byte != 255u;
    uneven = val && tid < left && static_cast<float>(d) < -kEvenSpan;
  }
  far = __syncthreads_or(far);
  uneven = __syncthreads_or(uneven);
  if (tid == 0) P.wide_far[(static_cast<long long>(val ? P.H : 0) + g) * gridDim.x + blk] = far;
  if (tid == 0)
    P.wide_scale[(static_cast<long long>(val ? P.H : 0) + g) * gridDim.x + blk] =
        val ? static_cast<float>(ref - 127) + (uneven ? kUnevenMark : 0.f) : e4m3_scale(ref);
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int x = i * kWidenThreads + tid, t = x / parts, pc = x - t * parts;
    if (x >= pieces || t >= left) continue;
    const __half2 f2 = *reinterpret_cast<const __half2 *>(&mult[t]);
    const uint32_t cw[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = e4m3x2_to_f16x2(cw[e]), hi = e4m3x2_to_f16x2_hi(cw[e]);
      const __half2 l2 = __hmul2(*reinterpret_cast<const __half2 *>(&lo), f2);
      const __half2 h2 = __hmul2(*reinterpret_cast<const __half2 *>(&hi), f2);
      o[2 * e] = *reinterpret_cast<const uint32_t *>(&l2);
      o[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&h2);
    }
    uint4 *const to = reinterpret_cast<uint4 *>(P.wide + ((static_cast<long long>(val ? P.P : 0) + tb + t) * P.H + g) * P.D * 2 + pc * 32);
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  grid_dependency_wait();  // over only after the mask kernel: the next kernel waits for this one alone
}

template <int CT, int DP, bool PRE>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
  using C = TileCfg<DP>;
  const int blocks = static_cast<int>(((PRE ? static_cast<long long>(p.B) : 1LL) * p.N * p.G + 255) / 256);
  const long long items = PRE ? static_cast<long long>(p.H) * blocks * p.psplits : static_cast<long long>(p.B) * p.H * blocks * p.osplits;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<attn_tile_kernel<CT, DP, PRE>>(C::kSmem, Roles<CT == SPEC_E4M3>::kLaunch);
  if (e != cudaSuccess) return e;
  // the mask and conversion kernels ahead of it let it start early
  return launch_after(attn_tile_kernel<CT, DP, PRE>, dim3(static_cast<unsigned>(items)), Roles<CT == SPEC_E4M3>::kThreads,
                      C::kSmem, s, p.first && (p.rowinfo || p.wide), p, blocks);
}

template <int CT>
cudaError_t launch_d(const AttnParams &p, bool prefix, cudaStream_t s) {
  if (p.D <= 64) return prefix ? launch<CT, 64, true>(p, s) : launch<CT, 64, false>(p, s);
  return prefix ? launch<CT, 128, true>(p, s) : launch<CT, 128, false>(p, s);
}

}  // namespace

cudaError_t launch_attn_widen(const AttnParams &p, cudaStream_t s) {
  const dim3 grid((p.P + kTok - 1) / kTok, p.H, 2);
  return launch_after(attn_widen_kernel, grid, kWidenThreads, 0, s, p.rowinfo != nullptr, p);
}

cudaError_t launch_attn_tile(const AttnParams &p, int ctype, bool prefix, cudaStream_t s) {
  if (ctype == SPEC_E4M3) return launch_d<SPEC_E4M3>(p, prefix, s);
  if (ctype == SPEC_BF16) return launch_d<SPEC_BF16>(p, prefix, s);
  return launch_d<SPEC_F16>(p, prefix, s);
}

}  // namespace sv
