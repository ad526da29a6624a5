// pages.cu -- the bookkeeping of a paged KV cache: block tables, the ring of
// free pages and slot maps (spec_page_plan), and the gather of an accepted tree
// path's entries across pages (spec_kv_compact_pages).
//
// The plan first reads the table and counts, per row, how many pages it wants and
// gives back; then it adds up the rows before each, moves pages between table and
// ring, and writes the slots.  Up to 256 rows that is one launch, else two.  What is taken
// (from the ring's head on) and what is given back (behind its tail) cannot
// overlap, since taken, free and given pages are at most the whole pool, so
// rows need not wait for one another.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"
#include "specverify.h"

namespace sv {
namespace {

constexpr int kPlThreads = 256;
constexpr int kPlWarps = kPlThreads / 32;  // rows per CTA
constexpr int kPlChunk = 8;                // places of a lane looked at together
// More slots per row than this are written by a whole CTA per row.
constexpr int kPlWide = 256;
// Up to so many rows are dealt with in one launch.
constexpr int kPlSmallThreads = 1024, kPlSmallCtas = 8;
constexpr int kPlSmallRows = kPlSmallCtas * kPlSmallThreads / 32;

struct PlanParams {
  int32_t *table, *free_pages, *free_state;
  const int32_t *kv_len, *count;
  int32_t *slot_map, *row_status;
  int32_t *state;         // workspace: {head, free pages} before the call; free pages < 0: not a ring's
  int2 *want;             // workspace [B]: pages taken and given back; x < 0: the row cannot be used
  int2 *sums;             // workspace [CTAs]: sums over their rows
  int B, N, columns, page, pages, window, sinks;
};

// Which of a row's places are live: below `need`, without [dead0, dead1).
struct Live {
  int need, dead0, dead1;
  __device__ __forceinline__ bool operator()(int j) const { return j < need && !(j >= dead0 && j < dead1); }
};
__device__ __forceinline__ bool row_live(const PlanParams &P, int b, int &n, int &c, Live &live) {
  n = __ldg(P.kv_len + b);
  c = P.count ? __ldg(P.count + b) : P.N;
  const long long total = static_cast<long long>(n) + c;
  if (n < 0 || c < 0 || c > P.N || total > static_cast<long long>(P.columns) * P.page) return false;
  live.need = static_cast<int>((total + P.page - 1) / P.page);
  live.dead0 = live.dead1 = 0;
  if (P.window > 0) {
    const int from = n - P.window + 1;  // tokens from here on are seen
    live.dead0 = P.sinks > 0x7fffffff - P.page ? 0x7fffffff : (P.sinks + P.page - 1) / P.page;
    live.dead1 = from > 0 ? from / P.page : 0;
  }
  return true;
}

// The ring's head and free pages (negative: not a ring's).
__device__ __forceinline__ int2 ring_state(const PlanParams &P) {
  const int head = P.free_state[0], have = P.free_state[1];
  const bool ok = head >= 0 && head < max(1, P.pages) && have >= 0 && have <= P.pages;
  return make_int2(head, ok ? have : -1);
}

// Pages that a row wants and gives back, by a warp; x < 0: it cannot be used.
__device__ __forceinline__ int2 count_row(const PlanParams &P, int b, int lane) {
  int n, c;
  Live live;
  if (!row_live(P, b, n, c, live)) return make_int2(-1, 0);
  bool ok = true;
  int2 want = make_int2(0, 0);
  const int32_t *const row = P.table + static_cast<size_t>(b) * P.columns;
  for (int j0 = lane; j0 < P.columns; j0 += 32 * kPlChunk) {
    int e[kPlChunk];
#pragma unroll
    for (int i = 0; i < kPlChunk; ++i) e[i] = j0 + i * 32 < P.columns ? row[j0 + i * 32] : -1;
#pragma unroll
    for (int i = 0; i < kPlChunk; ++i) {
      const int j = j0 + i * 32;
      ok = ok && e[i] < P.pages;
      if (j < P.columns) {
        const bool l = live(j);
        want.x += l && e[i] < 0;
        want.y += !l && e[i] >= 0;
      }
    }
  }
  want.x = __reduce_add_sync(FULL_MASK, want.x);
  want.y = __reduce_add_sync(FULL_MASK, want.y);
  return __all_sync(FULL_MASK, ok) ? want : make_int2(-1, 0);
}

__global__ void __launch_bounds__(kPlThreads) plan_count_kernel(const __grid_constant__ PlanParams P) {
  __shared__ int2 part[kPlWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = blockIdx.x * kPlWarps + warp;
  allow_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const int2 ring = ring_state(P);
    P.state[0] = ring.x;
    P.state[1] = ring.y;
  }
  int2 want = make_int2(0, 0);
  if (b < P.B) {
    want = count_row(P, b, lane);
    if (lane == 0) P.want[b] = want;
    if (want.x < 0) want = make_int2(0, 0);
  }
  if (lane == 0) part[warp] = want;
  __syncthreads();
  if (threadIdx.x == 0) {
    int2 s = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kPlWarps; ++w) s.x += part[w].x, s.y += part[w].y;
    P.sums[blockIdx.x] = s;
  }
}

// A warp moves a row's pages, behind what the rows before it take and give back;
// true: the ring was broken.
__device__ __forceinline__ bool move_pages(const PlanParams &P, int32_t *row, const Live &live, int head, int have, int2 before, bool served, int lane) {
  bool broken = false;
  int take = before.x, give = before.y;
  for (int j0 = 0; j0 < P.columns; j0 += 32) {
    const int j = j0 + lane;
    const int e = j < P.columns ? row[j] : -1;
    const bool l = live(j);
    const bool t = j < P.columns && l && e < 0 && served, g = j < P.columns && !l && e >= 0;
    const unsigned ts = __ballot_sync(FULL_MASK, t), gs = __ballot_sync(FULL_MASK, g), below = (1u << lane) - 1u;
    if (t) {
      const long long at = static_cast<long long>(head) + take + __popc(ts & below);
      const int page = P.free_pages[at % P.pages];
      const bool ok = page >= 0 && page < P.pages;
      if (ok) row[j] = page;
      broken = broken || !ok;
    }
    if (g) {
      const int rank = give + __popc(gs & below);
      if (rank < P.pages - have)
        P.free_pages[(static_cast<long long>(head) + have + rank) % P.pages] = e;
      else
        broken = true;
      row[j] = -1;
    }
    take += __popc(ts);
    give += __popc(gs);
  }
  return broken;
}
// The slots of a row's tokens i0, i0 + step, ...
__device__ __forceinline__ void write_slots(const PlanParams &P, int b, const int32_t *row, int n, int c, bool served, int i0, int step) {
  for (int i = i0; i < P.N; i += step) {
    int slot = -1;
    if (served && i < c) {
      const int t = n + i, j = t / P.page, e = row[j];
      if (e >= 0) slot = e * P.page + (t - j * P.page);
    }
    P.slot_map[static_cast<size_t>(b) * P.N + i] = slot;
  }
}

// Up to 256 rows in one launch: a cluster of CTAs with a warp per row, which tell
// one another what their rows want.  Bound by the host, which needs 15 us a call, 20
// with two launches; on the GPU 64 rows of 512 places take 5.0 us and 5.3, 128 of 2048
// 8.6 and 8.5, 200 of 512 6.7 and 5.6, 256 of 2048 11.3 and 8.5 (eight SMs' worth).
__global__ void __launch_bounds__(kPlSmallThreads) plan_small_kernel(const __grid_constant__ PlanParams P) {
  __shared__ int2 want[kPlSmallRows];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = blockIdx.x * (blockDim.x / 32) + warp;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int2 ring = ring_state(P);
  const int head = ring.x, have = ring.y;
  int2 w = make_int2(0, 0);
  if (b < P.B) w = count_row(P, b, lane);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others are running
  if (b < P.B) {
    if (lane < static_cast<int>(cluster_nctarank()))
      asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(dsmem_addr(&want[b], lane)), "r"(w.x), "r"(w.y) : "memory");
  }
  __syncwarp();
  cluster_sync();  // (also: everyone has read the ring)
  if (b < P.B) {
    int2 before = make_int2(0, 0);
    for (int i = lane; i < b; i += 32) {
      const int2 w = want[i];
      if (w.x >= 0) before.x += w.x, before.y += w.y;
    }
    before.x = __reduce_add_sync(FULL_MASK, before.x);
    before.y = __reduce_add_sync(FULL_MASK, before.y);
    const int2 mine = want[b];
    const bool usable = mine.x >= 0 && have >= 0, served = usable && (mine.x == 0 || before.x + mine.x <= have);
    int n = 0, c = 0;
    Live live = {};
    row_live(P, b, n, c, live);
    int32_t *const row = P.table + static_cast<size_t>(b) * P.columns;
    bool broken = false;
    if (usable && (mine.x > 0 || mine.y > 0)) broken = move_pages(P, row, live, head, have, before, served, lane);
    broken = __any_sync(FULL_MASK, broken);
    __syncwarp();
    if (lane == 0 && P.row_status) P.row_status[b] = !usable || broken ? SPEC_ROW_BAD_SLOT : !served ? SPEC_ROW_NO_PAGES : 0;
    write_slots(P, b, row, n, c, served, lane, 32);
  }
  // the ring after the call: what the rows up to the first that got nothing took
  if (blockIdx.x == 0 && warp == 0 && have >= 0 && P.pages > 0) {
    int taken = 0, given = 0;
    bool over = false;
    for (int i0 = 0; i0 < P.B; i0 += 32) {
      const int2 w = i0 + lane < P.B ? want[i0 + lane] : make_int2(0, 0);
      given += __reduce_add_sync(FULL_MASK, w.x >= 0 ? w.y : 0);
      int x = max(w.x, 0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, x, o);
        if (lane >= o) x += y;
      }
      if (over) continue;
      const unsigned beyond = __ballot_sync(FULL_MASK, taken + x > have);
      over = beyond != 0;
      const int k = over ? __ffs(beyond) - 2 : 31;  // the last that was served
      if (k >= 0) taken += __shfl_sync(FULL_MASK, x, k);
    }
    if (lane == 0) {
      P.free_state[0] = static_cast<int>((static_cast<long long>(head) + taken) % P.pages);
      P.free_state[1] = have - taken + min(given, P.pages - have);
    }
  }
}

// WIDE: a CTA per row, whose first warp does the table; else a warp per row.
template <bool WIDE>
__global__ void __launch_bounds__(kPlThreads) plan_apply_kernel(const __grid_constant__ PlanParams P) {
  __shared__ int2 part[kPlWarps];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int b0 = WIDE ? blockIdx.x : blockIdx.x * kPlWarps;  // the CTA's first row
  const int b = WIDE ? b0 : b0 + warp;
  grid_dependency_wait();
  // --- what the rows before this CTA's take and give back
  const int head = P.state[0], have = P.state[1];
  int2 before = make_int2(0, 0);
  const int group = b0 / kPlWarps;
  for (int i = tid; i < group; i += kPlThreads) {
    const int2 s = P.sums[i];
    before.x += s.x, before.y += s.y;
  }
  if (WIDE && tid < b0 - group * kPlWarps) {
    const int2 s = P.want[group * kPlWarps + tid];
    if (s.x >= 0) before.x += s.x, before.y += s.y;
  }
  before.x = __reduce_add_sync(FULL_MASK, before.x);
  before.y = __reduce_add_sync(FULL_MASK, before.y);
  if (lane == 0) part[warp] = before;
  __syncthreads();
  before = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kPlWarps; ++w) before.x += part[w].x, before.y += part[w].y;
  const int last_row = min(P.B, WIDE ? b0 + 1 : b0 + kPlWarps) - 1;
  int2 mine = b < P.B ? P.want[b] : make_int2(0, 0);
  const bool usable = b < P.B && mine.x >= 0 && have >= 0;
  if (mine.x < 0) mine = make_int2(0, 0);
  if (!WIDE)
    for (int w = 0; w < warp; ++w)
      if (b0 + w < P.B) {
        const int2 s = P.want[b0 + w];
        if (s.x >= 0) before.x += s.x, before.y += s.y;
      }
  const int upto = before.x + mine.x;  // wanted up to and with this row
  const bool served = usable && (mine.x == 0 || upto <= have);
  bool broken = false;
  int n = 0, c = 0;
  Live live = {};
  if (b < P.B) row_live(P, b, n, c, live);
  int32_t *const row = P.table + static_cast<size_t>(b) * P.columns;
  if (usable && (mine.x > 0 || mine.y > 0) && (!WIDE || warp == 0)) broken = move_pages(P, row, live, head, have, before, served, lane);
  if (WIDE) {
    broken = __syncthreads_or(broken);  // also: the table's changes are seen by the whole CTA
  } else {
    broken = __any_sync(FULL_MASK, broken);
    __syncwarp();
  }
  if (b < P.B) {
    const bool lead = WIDE ? tid == 0 : lane == 0;
    if (lead && P.row_status)
      P.row_status[b] = !usable || broken ? SPEC_ROW_BAD_SLOT : !served ? SPEC_ROW_NO_PAGES : 0;
    write_slots(P, b, row, n, c, served, WIDE ? tid : lane, WIDE ? kPlThreads : 32);
  }
  // --- the ring after the call, by the CTA of the last row: all that was wanted,
  // or where that is too much what the rows up to the first that got nothing took
  if (last_row == P.B - 1 && have >= 0 && warp == (WIDE ? 0 : last_row - b0)) {
    int taken = upto;
    if (taken > have) {
      int run = 0, g0 = 0;
      const int groups = (P.B + kPlWarps - 1) / kPlWarps;
      for (; g0 < groups; g0 += 32) {
        int x = g0 + lane < groups ? P.sums[g0 + lane].x : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULL_MASK, x, o);
          if (lane >= o) x += y;
        }
        const unsigned over = __ballot_sync(FULL_MASK, run + x > have);
        if (over) {
          const int k = __ffs(over) - 1;
          if (k > 0) run += __shfl_sync(FULL_MASK, x, k - 1);
          g0 += k;
          break;
        }
        run += __shfl_sync(FULL_MASK, x, 31);
      }
      for (int r = g0 * kPlWarps; r < min(P.B, (g0 + 1) * kPlWarps); ++r) {
        const int x = max(P.want[r].x, 0);
        if (run + x > have) break;
        run += x;
      }
      taken = run;
    }
    if (lane == 0 && P.pages > 0) {
      const int given = min(before.y + mine.y, P.pages - have);
      P.free_state[0] = static_cast<int>((static_cast<long long>(head) + taken) % P.pages);
      P.free_state[1] = have - taken + given;
    }
  }
}

// ------------------------------------------------------------- compaction
constexpr int kPcThreads = 128;  // 16-byte columns per CTA
constexpr int kPcBatch = 8;      // path entries loaded before they are stored
constexpr int kPcPath = 64;      // path entries whose places are looked up together

struct CompactParams {
  unsigned char *kv;
  long long E, plane_stride, page_stride, tok_stride;
  const int32_t *table, *kv_len, *accepted_len, *path_nodes;
  int32_t *row_status;
  int B, N, columns, page, pages;
};

// Where token t of a row is, relative to its plane; negative: on no page.
__device__ __forceinline__ long long place(const CompactParams &P, const int32_t *row, int t) {
  const int j = t / P.page, g = __ldg(row + j);
  if (g < 0 || g >= P.pages) return -1;
  return g * P.page_stride + (t - j * P.page) * P.tok_stride;
}

// The moves are safe in place in this order: path node k is token >= k + 1 of
// the pass (the path increases strictly), so a later entry's source is never a
// place that was written before it is read, and within a batch every source is
// read before any place is written.  Bound by latency (two dependent look-ups
// before the first byte) on small paths, else by HBM.
__global__ void __launch_bounds__(kPcThreads) kv_compact_pages_kernel(const __grid_constant__ CompactParams P) {
  const int b = blockIdx.z, p = blockIdx.y, tid = threadIdx.x;
  __shared__ long long from[kPcPath], to[kPcPath];
  const int a = __ldg(P.accepted_len + b), base = __ldg(P.kv_len + b);
  const int32_t *const path = P.path_nodes + static_cast<size_t>(b) * P.N;
  const int32_t *const row = P.table + static_cast<size_t>(b) * P.columns;
  bool increasing = true, placed = true;
  if (a > 0) {
    increasing = a <= P.N - 1;
    for (int k = tid; increasing && k < a; k += kPcThreads) {
      const int n = __ldg(path + k), prev = k == 0 ? 0 : __ldg(path + k - 1);
      if (n <= prev || n >= P.N) {
        increasing = false;
      } else if (base < 0 || static_cast<long long>(base) + n >= static_cast<long long>(P.columns) * P.page) {
        placed = false;
      } else {  // base + 1 + k <= base + n
        const long long f = place(P, row, base + n), t = place(P, row, base + 1 + k);
        placed = placed && f >= 0 && t >= 0;
        if (k < kPcPath) from[k] = f, to[k] = t;
      }
    }
  }
  increasing = __syncthreads_and(increasing);
  placed = __syncthreads_and(placed);
  if (tid == 0 && blockIdx.x == 0 && p == 0 && P.row_status)
    P.row_status[b] = !increasing ? SPEC_ROW_BAD_PARENT : !placed ? SPEC_ROW_BAD_SLOT : 0;
  if (!increasing || !placed || a <= 0) return;
  const long long col = static_cast<long long>(blockIdx.x) * kPcThreads + tid;
  const bool on = col * 16 < P.E;
  unsigned char *const at = P.kv + p * P.plane_stride + col * 16;
  for (int c0 = 0; c0 < a; c0 += kPcPath) {
    if (c0 > 0) {
      __syncthreads();
      for (int k = tid; k < min(kPcPath, a - c0); k += kPcThreads) {
        from[k] = place(P, row, base + __ldg(path + c0 + k));
        to[k] = place(P, row, base + 1 + c0 + k);
      }
      __syncthreads();
    }
    if (!on) continue;
    const int n = min(kPcPath, a - c0);
    for (int k0 = 0; k0 < n; k0 += kPcBatch) {
      uint4 v[kPcBatch];
#pragma unroll
      for (int i = 0; i < kPcBatch; ++i)
        if (k0 + i < n) v[i] = *reinterpret_cast<const uint4 *>(at + from[k0 + i]);
#pragma unroll
      for (int i = 0; i < kPcBatch; ++i)
        if (k0 + i < n) *reinterpret_cast<uint4 *>(at + to[k0 + i]) = v[i];
    }
  }
}

bool pg_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t pg_round(size_t x) { return (x + 255) / 256 * 256; }
int groups_of(int B) { return (B + kPlWarps - 1) / kPlWarps; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_page_plan_workspace_size(int32_t B) {
  if (B < 0 || B > 1 << 20) return 0;
  return 256 + pg_round(static_cast<size_t>(B) * sizeof(int2)) + pg_round(static_cast<size_t>(groups_of(B)) * sizeof(int2));
}

spec_status spec_page_plan(const spec_page_plan_args *a, int32_t *slot_map, int32_t *row_status, void *ws,
                           size_t ws_bytes, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const long long most = 0x7fffffffLL;
  if (a->B < 0 || a->B > 1 << 20 || a->N < 0 || a->columns < 1 || a->page_size < 16 || a->page_size > SPEC_MAX_PAGE ||
      a->page_size % 16 || a->num_pages < 0)
    return SPEC_ERR_SHAPE;
  if (static_cast<long long>(a->columns) * a->page_size > most || static_cast<long long>(a->num_pages) * a->page_size > most ||
      static_cast<long long>(a->B) * a->N > most || static_cast<long long>(a->B) * a->columns > most)
    return SPEC_ERR_SHAPE;
  if (a->window < 0 || a->sinks < 0) return SPEC_ERR_ARG;
  if (a->B == 0) return SPEC_OK;
  const void *w4[] = {a->block_table, a->free_pages, a->free_state, a->kv_len, a->count, slot_map, row_status};
  for (const void *q : w4)
    if (!pg_aligned(q, 4)) return SPEC_ERR_ALIGN;
  if (!a->block_table || !a->free_state || !a->kv_len || (a->num_pages > 0 && !a->free_pages) || (a->N > 0 && !slot_map))
    return SPEC_ERR_NULL;
  if (!ws || !pg_aligned(ws, 256) || ws_bytes < spec_page_plan_workspace_size(a->B)) return SPEC_ERR_WORKSPACE;
  char *w = static_cast<char *>(ws);
  PlanParams p = {};
  p.table = a->block_table;
  p.free_pages = a->free_pages;
  p.free_state = a->free_state;
  p.kv_len = a->kv_len;
  p.count = a->count;
  p.slot_map = slot_map;
  p.row_status = row_status;
  p.state = reinterpret_cast<int32_t *>(w);
  p.want = reinterpret_cast<int2 *>(w + 256);
  p.sums = reinterpret_cast<int2 *>(w + 256 + pg_round(static_cast<size_t>(a->B) * sizeof(int2)));
  p.B = a->B;
  p.N = a->N;
  p.columns = a->columns;
  p.page = a->page_size;
  p.pages = a->num_pages;
  p.window = a->window;
  p.sinks = a->sinks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->B <= kPlSmallRows && a->N <= kPlWide) {
    const int ctas = std::min(a->B, kPlSmallCtas), rows = (a->B + ctas - 1) / ctas;  // spread over as many SMs as go
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * rows);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_small_kernel, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }
  const int groups = groups_of(a->B);
  plan_count_kernel<<<groups, kPlThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  const cudaError_t e = a->N > kPlWide ? launch_after(plan_apply_kernel<true>, dim3(a->B), kPlThreads, 0, s, true, p)
                                       : launch_after(plan_apply_kernel<false>, dim3(groups), kPlThreads, 0, s, true, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_compact_pages(const spec_page_compact_args *a, int32_t *row_status, void *stream) {
  if (!a) return SPEC_ERR_NULL;
  const long long most = 0x7fffffffLL;
  if (a->B < 0 || a->B > 65535 || a->planes < 0 || a->planes > 65535 || a->N < 1 || a->N > SPEC_MAX_TREE_NODES || a->columns < 1 ||
      a->page_size < 16 || a->page_size > SPEC_MAX_PAGE || a->page_size % 16 || a->num_pages < 0 || a->entry_bytes < 0 ||
      a->entry_bytes > most || a->plane_stride < 0 || a->page_stride < 0 || a->tok_stride < 0)
    return SPEC_ERR_SHAPE;
  if (static_cast<long long>(a->columns) * a->page_size > most || static_cast<long long>(a->num_pages) * a->page_size > most)
    return SPEC_ERR_SHAPE;
  if (!pg_aligned(a->kv, 16) || a->entry_bytes % 16 || a->plane_stride % 16 || a->page_stride % 16 || a->tok_stride % 16)
    return SPEC_ERR_ALIGN;
  const void *w4[] = {a->block_table, a->kv_len_in, a->accepted_len, a->path_nodes, row_status};
  for (const void *q : w4)
    if (!pg_aligned(q, 4)) return SPEC_ERR_ALIGN;
  if (a->B == 0) return SPEC_OK;
  if (!a->block_table || !a->kv_len_in || !a->accepted_len || !a->path_nodes ||
      (!a->kv && a->num_pages > 0 && a->planes > 0 && a->entry_bytes > 0))
    return SPEC_ERR_NULL;
  CompactParams p = {};
  p.kv = static_cast<unsigned char *>(a->kv);
  p.E = a->entry_bytes;
  p.plane_stride = a->plane_stride;
  p.page_stride = a->page_stride;
  p.tok_stride = a->tok_stride;
  p.table = a->block_table;
  p.kv_len = a->kv_len_in;
  p.accepted_len = a->accepted_len;
  p.path_nodes = a->path_nodes;
  p.row_status = row_status;
  p.B = a->B;
  p.N = a->N;
  p.columns = a->columns;
  p.page = a->page_size;
  p.pages = a->num_pages;
  // with no entries to move the rows' checks run all the same
  const long long chunks = (a->entry_bytes / 16 + kPcThreads - 1) / kPcThreads;
  if (a->planes == 0) p.E = 0;
  const dim3 grid(static_cast<unsigned>(chunks > 0 ? chunks : 1), a->planes > 0 ? a->planes : 1, a->B);
  kv_compact_pages_kernel<<<grid, kPcThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
