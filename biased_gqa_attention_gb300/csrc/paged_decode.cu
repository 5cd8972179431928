// paged_decode.cu -- attention of one new token per sequence over a cache in
// pages.
//
// Bound: HBM.  Every live K and V row is read once per unit: a (sequence, KV head,
// group of query heads), 4 D bytes a key in bf16 for 4 D flops a head.  A group
// is all heads of a KV head up to 8, or 16 (unit_rows()); a KV head with more has
// several units, which read its rows again: two sequences of
// 131071 and one KV head of 128, 37.8 us with 16 query heads and 85.4 with 64; of
// 65536 and 512, 65.5 us with 8 and 92.8 with 16.
//
// The batch's work is one axis of tiles (KT keys of one unit), unit after unit.
// Every CTA takes an equal contiguous slice of it and every warp an equal part of
// that, whatever the sequences' lengths are: a warp works through its part by
// a ring of shared-memory slots of its own, so warps do not wait for each other
// while they stream.  The tensor-core kernels' rings are filled by a producer warp
// (TMA boxes of page rows; page sizes that are multiples of 16); for other page
// sizes, and on the SIMT lanes, a warp copies its own rows (16-byte cp.async, a
// row's address from the page table, rows outside the sequence filled with zeros),
// and a page may end anywhere in a tile.  A unit
// that lies in one warp's part is written out by it; a unit split over warps of
// a CTA is joined by the CTA at its end, and one split over CTAs by the merge
// kernel, from each CTA's (max, sum, unnormalised output) in the workspace.
// Everything is joined in the order of the axis, so the result does not depend
// on timing.
//
// Measured (GB300, cold L2; the copy rate is 6.78 TB/s): 32 sequences of 1 to 8192
// keys, 2 KV heads of 512 (467 MB): 91 us, 5.1 TB/s; three sequences of 131071, 65537
// and 12345, 2 KV heads of 128 (214 MB): 47 us, 4.6 TB/s; one sequence of 517, 8 KV
// heads of 256, on a cluster per unit: 9.7 us (its 4 MB take 0.6).  Two CTAs an SM
// (94 and 49 us on the first two) and four to six waves of smaller CTAs (102 to
// 106 and 61 to 63 us) were slower: each CTA pays its start and its join.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "simt_tile.cuh"
#include "tma_host.h"

namespace extkv {

namespace {

constexpr uint32_t kWaitPolls = 1u << 22;  // bounded waits
constexpr int kMaxCluster = 8;

struct PagedParams {
  void* y;
  const void* q;
  const void* k;
  const void* v;
  const int64_t* table;
  const int64_t* nonpad;
  float c;  // scale * log2(e)
  int window, B, Hq, Hkv, g, D, page_size, max_pages;
  int64_t num_pages, q_stride;
  int box;     // rows of a TMA request
  int cluster; // CTAs of a unit's cluster (cluster kernel)
  uint32_t wait_limit;
  int rows;    // query heads per unit (the kernel's row capacity)
  int groups;  // units per (sequence, KV head)
  int units;   // groups * Hkv: units of a sequence
  int slices;     // pieces the axis is cut into that the merge kernel joins: CTAs (tensor cores) or warps
  int64_t* base;  // [B + 1] tiles before each sequence (per unit of it)
  float2* ml;     // [slices][2][rows] (max in log2 units, sum)
  float* part;    // [slices][2][rows][D]
  float2* w_ml;   // [slices][warps][rows]: partials a CTA joins itself
  float* w_part;  // [slices][warps][rows][D]
  int32_t* status;
};

struct LiveKeys {
  int lo, hi;
};

__device__ __forceinline__ int64_t length_of(const PagedParams& p, int b) {
  return EXTKV_IN_KIND(kChkLens, b, 1, p.B, p.status) ? p.nonpad[b] : 0;
}

// The pool's page that holds sequence b's slots from pg * page_size on.
__device__ __forceinline__ int64_t page_of(const PagedParams& p, int b, int pg) {
  const int64_t at = static_cast<int64_t>(b) * p.max_pages + pg;
  return EXTKV_IN_KIND(kChkTable, at, 1, static_cast<int64_t>(p.B) * p.max_pages, p.status) ? p.table[at] : -1;
}

// Elements from q's, y's, the partials' start (checked builds).
__device__ __forceinline__ bool q_in(const PagedParams& p, int64_t first) {
  return EXTKV_IN_KIND(kChkRows, first, p.D, (p.B - 1) * p.q_stride + static_cast<int64_t>(p.Hq) * p.D, p.status);
}
__device__ __forceinline__ bool y_in(const PagedParams& p, int64_t first, int count) {
  return EXTKV_IN_KIND(kChkOut, first, count, static_cast<int64_t>(p.B) * p.Hq * p.D, p.status);
}
__device__ __forceinline__ bool base_in(const PagedParams& p, int b) {
  return EXTKV_IN_KIND(kChkPartial, b, 1, static_cast<int64_t>(p.B) + 1, p.status);
}
// rows at .. of ml and part, which have `sets` times p.rows
__device__ __forceinline__ bool part_in(const PagedParams& p, int64_t at, int rows, int64_t sets) {
  return EXTKV_IN_KIND(kChkPartial, at, rows, sets * p.rows, p.status);
}

__device__ __forceinline__ LiveKeys live_keys(const PagedParams& p, int b) {
  const int64_t np = length_of(p, b);
  if (np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size) return {0, 0};
  const int n = static_cast<int>(np);
  return {p.window > 0 && n > p.window ? n - p.window : 0, n};
}

// Tiles start at multiples of KT.
template <int KT>
__device__ __forceinline__ int tiles_of(LiveKeys k) {
  return k.lo < k.hi ? (k.hi + KT - 1) / KT - k.lo / KT : 0;
}

// The axis of tiles cut into slices: p.slices, or one per tile when there are
// fewer; the first `more` of them hold one tile more than the others.
struct Axis {
  int64_t total, each;
  int n, more;
  __device__ __forceinline__ Axis(const PagedParams& p, int64_t total_) : total(total_) {
    n = total < p.slices ? static_cast<int>(total) : p.slices;
    each = n ? div(total, n) : 0;
    more = static_cast<int>(total - each * n);
  }
  __device__ __forceinline__ int64_t start(int i) const { return i * each + min(i, more); }
  // the slice that holds tile f
  __device__ __forceinline__ int holds(int64_t f) const {
    const int64_t cut = more * (each + 1);
    return static_cast<int>(f < cut ? div(f, each + 1) : more + div(f - cut, each));
  }
  // 64-bit division costs some hundred instructions: not where 32 bits do
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
  }
};

// A position on the axis of tiles.
template <int KT>
struct Cursor {
  int b, u, t, tiles;
  LiveKeys keys;
  // the tile's first key
  __device__ __forceinline__ int key0() const { return (keys.lo / KT + t) * KT; }
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++t < tiles) return;
    t = 0;
    if (++u < p.units) return;
    u = 0;
    do {
      if (++b >= p.B) return;
      keys = live_keys(p, b);
      tiles = tiles_of<KT>(keys);
    } while (tiles == 0);
  }
};

// Block-wide: the tiles before each chunk of sequences, and their total.  Block
// 0 also leaves every sequence's base for the merge kernel and flags lengths
// outside the table.  `pre` has blockDim.x + 1 entries.
template <int KT>
__device__ __forceinline__ int scan_tiles(const PagedParams& p, int64_t* pre, int64_t* warp_sum) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + nt - 1) / nt;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += tiles_of<KT>(live_keys(p, b));
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t off = 0;
  for (int w = 0; w < warp; ++w) off += warp_sum[w];
  pre[tid] = off + inc - sum;
  if (tid == nt - 1) pre[nt] = off + inc;
  __syncthreads();
  if (blockIdx.x == 0) {
    int64_t at = pre[tid];
    for (int b = b0; b < b1; ++b) {
      if (base_in(p, b)) p.base[b] = at;
      at += tiles_of<KT>(live_keys(p, b));
      const int64_t np = length_of(p, b);
      if (np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size) report(p.status, EXTKV_DEV_BAD_NONPAD);
    }
    if (tid == nt - 1 && base_in(p, p.B)) p.base[p.B] = pre[nt];
  }
  return per;
}

// The cursor at tile f of the axis (f < total); the warp's lanes search together.
template <int KT>
__device__ __forceinline__ Cursor<KT> cursor_at(const PagedParams& p, const int64_t* pre, int per, int64_t f) {
  // the last chunk of sequences whose first tile is <= f: 32 candidates at a time
  const int lane = threadIdx.x & 31, chunks = blockDim.x, step = (chunks + 31) / 32;
  const int wide = __popc(__ballot_sync(0xffffffffu, lane * step < chunks && pre[lane * step] * p.units <= f)) - 1;
  const int at = wide * step + lane;
  const int chunk = wide * step + __popc(__ballot_sync(0xffffffffu, lane < step && at < chunks && pre[at] * p.units <= f)) - 1;
  int64_t rest = f - pre[chunk] * p.units;
  Cursor<KT> c;
  c.b = chunk * per;
  for (;;) {
    c.keys = live_keys(p, c.b);
    c.tiles = tiles_of<KT>(c.keys);
    const int64_t n = static_cast<int64_t>(c.tiles) * p.units;
    if (rest < n) break;
    rest -= n;
    ++c.b;
  }
  c.u = static_cast<int>(Axis::div(rest, c.tiles));
  c.t = static_cast<int>(rest - static_cast<int64_t>(c.u) * c.tiles);
  return c;
}

// The same for at most 32 sequences, a lane each: every warp scans them for
// itself, without meeting the block and without loading a length twice.
template <int KT>
struct LaneScan {
  LiveKeys keys;
  int64_t end;  // tiles (per unit) up to and with this lane's sequence
  __device__ __forceinline__ explicit LaneScan(const PagedParams& p) {
    const int lane = threadIdx.x & 31;
    const int64_t np = lane < p.B ? length_of(p, lane) : 0;
    const bool bad = np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size;
    const int n = bad ? 0 : static_cast<int>(np);
    keys = {p.window > 0 && n > p.window ? n - p.window : 0, n};
    const int64_t mine = tiles_of<KT>(keys);
    end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    if (p.B <= 32 && blockIdx.x == 0 && threadIdx.x < 32) {
      if (lane < p.B && base_in(p, lane)) p.base[lane] = end - mine;
      if (lane == 31 && base_in(p, p.B)) p.base[p.B] = end;
      if (bad) report(p.status, EXTKV_DEV_BAD_NONPAD);
    }
  }
  __device__ __forceinline__ int64_t total(const PagedParams& p) const {
    return __shfl_sync(0xffffffffu, end, 31) * p.units;
  }
  // f is the warp's
  __device__ __forceinline__ Cursor<KT> cursor_at(const PagedParams& p, int64_t f) const {
    Cursor<KT> c;
    c.b = __popc(__ballot_sync(0xffffffffu, end * p.units <= f));
    c.keys.lo = __shfl_sync(0xffffffffu, keys.lo, c.b);
    c.keys.hi = __shfl_sync(0xffffffffu, keys.hi, c.b);
    c.tiles = tiles_of<KT>(c.keys);
    const int64_t rest = f - (__shfl_sync(0xffffffffu, end, c.b) - c.tiles) * p.units;
    c.u = static_cast<int>(Axis::div(rest, c.tiles));
    c.t = static_cast<int>(rest - static_cast<int64_t>(c.u) * c.tiles);
    return c;
  }
};

// Pool rows of a tile, one per lane: the page id is loaded a tile ahead.
template <int KT>
struct TileRows {
  int64_t page;
  int off, u;
  bool live, lead;  // lead: the page's first live row of this tile
  __device__ __forceinline__ void look_up(const PagedParams& p, const Cursor<KT>& c) {
    const int lane = threadIdx.x & 31;
    const int j = c.key0() + lane;
    live = lane < KT && j >= c.keys.lo && j < c.keys.hi;
    u = c.u;
    off = 0;
    page = -1;
    lead = false;
    if (live) {
      const int pg = j / p.page_size;
      off = j - pg * p.page_size;
      lead = lane == 0 || off == 0 || j == c.keys.lo;
      page = page_of(p, c.b, pg);
    }
  }
  // row of the pool in units of D elements, or ~0
  __device__ __forceinline__ uint32_t row(const PagedParams& p) const {
    if (!live) return ~0u;
    if (page < 0 || page >= p.num_pages) {
      if (u == 0 && lead) report(p.status, EXTKV_DEV_BAD_PAGE);
      return ~0u;
    }
    const int64_t r = (page * p.Hkv + u / p.groups) * p.page_size + off;
    if (!EXTKV_IN_KIND(kChkPages, r, 1, p.num_pages * p.Hkv * p.page_size, p.status)) return ~0u;
    return static_cast<uint32_t>(r);
  }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- tensor cores (bf16) -----------------------------------------------------------
// S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16: 16 keys (or 16 columns
// of V) by 8 query heads, so that up to 8 heads cost one pass and the softmax's
// maximum and sum are per column.  The path is bound by HBM: its products need
// about 8 flops a byte, a few percent of the tensor pipe, and tcgen05's 128 rows
// would be mostly padding.
//
// A consumer warp has a ring of slots that hold K and V tiles in turn (KT keys
// each, 64-column chunks of 128-byte swizzled rows), so that a slot is refilled
// as soon as its one product is done.  Two ways to fill it:
//   TMA   pages of whole boxes (page_size a multiple of 16): a producer warp,
//         one lane per consumer, issues one request for a box of 16 or KT rows.
//         The consumers then execute no load instructions: a few warps a
//         scheduler hold the whole register file, and a tile's instructions
//         should take no longer than its bytes.
//   else  any other page size: the consumer's lanes copy 16 bytes each
//         (cp.async), a row's address from the page table.

// Few short units (a small batch, a sliding window) leave the joining of CTAs as
// a good part of the call.  There a cluster of CTAs takes one unit, each CTA an
// equal share of its tiles, and the shares are joined through distributed shared
// memory in rank order: one launch, no scan of the batch, no workspace.

// Rings and warps by head size, of those that fit: six warps, or four where
// sixteen heads' accumulators (D/4 a thread and eight heads) fill the registers; tiles of
// 32 keys while a ring still holds four of them.  Against one slice per warp without a
// producer, all joined by the merge kernel: 59 to 47 us on the long sequences above.
template <int D_, int NT_, int KT_, int SLOTS_, int WARPS_, bool TMA_, bool CLUSTER_ = false>
struct MmaCfg {
  static constexpr int D = D_, NT = NT_, KT = KT_, SLOTS = SLOTS_, WARPS = WARPS_;
  static constexpr bool TMA = TMA_, CLUSTER = CLUSTER_;
  static constexpr int kThreads = (WARPS + (TMA ? 1 : 0)) * 32;
  static constexpr int kTile = KT * D * 2;  // a slot
  static constexpr int kRing = SLOTS * kTile;
  static constexpr int kShare = CLUSTER ? 8 * NT * (D * 4 + 8) : 0;  // a CTA's joined partial
  static constexpr int kSmem = WARPS * kRing + kShare + 1024;
};

// What a warp leaves to its CTA: the units its part begins [0] and ends [1] in,
// whether the first was left early (to the workspace) and the last late (in the
// ring), and whether the late one begins and ends its unit.
struct Rec {
  int n, early, late, begins, ends;
  int b[2], u[2];
};

// Partials of one unit in a CTA: late ones of the warps in `members`, then the
// early one of warp `early` (-1: none).
struct Chain {
  unsigned members;
  int early, b, u, whole, slot;
};

// Bounded wait: polls first (the warp has its scheduler almost to itself), then
// suspends; gives up once another warp has.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit) {
  uint32_t i = 0;
  for (; i < limit && i < 64; ++i)
    if (ptx::mbar_test_wait(bar, parity)) return true;
  for (; i < limit; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 127u) == 127u && *abort) return false;
  }
  *abort = 1;
  return false;
}

// Bits of the keys [lo, hi) in a tile of KT keys that starts at k0.
template <int KT>
__device__ __forceinline__ uint32_t key_bits(int lo, int hi, int k0) {
  const int a = max(lo - k0, 0), b = min(hi - k0, KT);
  if (a >= b) return 0;
  return (b >= 32 ? ~0u : (1u << b) - 1u) & (~0u << a);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    paged_decode_mma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                            const PagedParams p) {
  constexpr int D = C::D, NT = C::NT, KT = C::KT, NS = C::SLOTS, KS = KT / 16, W = C::WARPS;
  constexpr int kRowsU = 8 * NT;
  constexpr int kPad = D + 4;  // rows of a partial in shared memory start in different banks
  constexpr uint32_t kFull = KT == 32 ? ~0u : (1u << (KT & 31)) - 1u;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t pre[C::kThreads + 1], warp_sum[C::kThreads / 32];
  __shared__ uint32_t live_mask[W][NS];  // keys of the slot's K tile that were loaded
  __shared__ Rec rec[W];
  __shared__ Chain chains[W + 1];
  __shared__ int n_chains;
  __shared__ uint64_t full[W][NS], empty[W][NS];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane >> 2, qi = lane & 3;
  if (C::TMA) {
    for (int i = tid; i < W * NS; i += C::kThreads) {
      ptx::mbar_init(&full[i / NS][i % NS], 1);
      ptx::mbar_init(&empty[i / NS][i % NS], 1);
    }
    if (tid == 0) {
      abort_flag = 0;
      ptx::prefetch_tensormap(&kmap);
      ptx::prefetch_tensormap(&vmap);
    }
    ptx::fence_mbar_init();
  }
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int cta = blockIdx.x;
  Cursor<KT> cur{};
  int n, mine = C::TMA && warp == W ? min(lane, W - 1) : warp;  // a consumer's part; the producer's lanes serve one each
  int unit_tiles = 0, tiles_here = 0, rank = 0;
  if constexpr (C::CLUSTER) {
    __syncthreads();  // the barriers
    rank = static_cast<int>(ptx::cluster_ctarank());
    const int unit = cta / p.cluster;
    cur.b = unit / p.units;
    cur.u = unit - cur.b * p.units;
    const int64_t np = length_of(p, cur.b);
    if (tid == 0 && rank == 0 && cur.u == 0 && (np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size))
      report(p.status, EXTKV_DEV_BAD_NONPAD);
    cur.keys = live_keys(p, cur.b);
    cur.tiles = unit_tiles = tiles_of<KT>(cur.keys);
    const int t0 = static_cast<int>(static_cast<int64_t>(unit_tiles) * rank / p.cluster);
    tiles_here = static_cast<int>(static_cast<int64_t>(unit_tiles) * (rank + 1) / p.cluster) - t0;
    auto first_of = [&](int w) { return static_cast<int>(static_cast<int64_t>(tiles_here) * w / W); };
    cur.t = t0 + first_of(mine);
    n = first_of(mine + 1) - first_of(mine);
  } else {
    const bool few = p.B <= 32;
    const LaneScan<KT> scan(p);  // (of the first 32 sequences where there are more: not used)
    int per = 0;
    if (few) __syncthreads();  // the barriers
    else per = scan_tiles<KT>(p, pre, warp_sum);
    const Axis axis(p, few ? scan.total(p) : pre[blockDim.x] * p.units);
    if (cta >= axis.n) return;
    const int64_t c0 = axis.start(cta);
    tiles_here = static_cast<int>(axis.start(cta + 1) - c0);  // at least one
    auto first_of = [&](int w) { return static_cast<int>(static_cast<int64_t>(tiles_here) * w / W); };
    auto at_tile = [&](int64_t f) { return few ? scan.cursor_at(p, f) : cursor_at<KT>(p, pre, per, f); };
    if (!C::TMA || warp < W) {
      if (first_of(mine) < first_of(mine + 1)) cur = at_tile(c0 + first_of(mine));
    } else {
      for (int w = 0; w < W; ++w)
        if (first_of(w) < first_of(w + 1)) {
          const Cursor<KT> c = at_tile(c0 + first_of(w));
          if (w == mine) cur = c;
        }
    }
    n = first_of(mine + 1) - first_of(mine);
  }

  if (C::TMA && warp == W) {
    // ---------------- producer ----------------
    uint8_t* ring = smem + mine * C::kRing;
    const int boxes = KT / p.box;  // per tile: 1, or 2
    int64_t page[2];
    int off[2];
    auto look_up = [&] {  // the tile's pages; -2: not needed
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = cur.key0() + x * p.box, pg = j / p.page_size;
        off[x] = j - pg * p.page_size;
        page[x] = -2;
        if (x < boxes && j < cur.keys.hi && j + p.box > cur.keys.lo)
          page[x] = page_of(p, cur.b, pg);
      }
    };
    const int groups = lane < W ? 2 * n : 0;  // K, V, K, V, ...
    if (groups) look_up();
    int g = 0, slot = 0, phase = 1;  // phase: of the empty barrier to wait for (none in the first round)
    uint32_t idle = 0;
    bool stop = false;
    while (!stop && __any_sync(0xffffffffu, g < groups)) {
      const bool can = g < groups && (g < NS || ptx::mbar_test_wait(&empty[mine][slot], phase));
      if (can) {
        const CUtensorMap* map = (g & 1) ? &vmap : &kmap;
        uint8_t* dst = ring + slot * C::kTile;
        uint32_t mask = 0, bytes = 0;
        int row[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          row[x] = -1;
          if (page[x] == -2) continue;
          if (page[x] < 0 || page[x] >= p.num_pages) {
            if (cur.u == 0 && !(g & 1)) report(p.status, EXTKV_DEV_BAD_PAGE);
            continue;
          }
          row[x] = static_cast<int>(page[x] * p.Hkv + cur.u / p.groups);
          bytes += p.box * D * 2;
          mask |= (p.box == 32 ? ~0u : (1u << p.box) - 1u) << (x * p.box);
        }
        live_mask[mine][slot] = mask;
        if (bytes) {
          ptx::mbar_arrive_expect_tx(&full[mine][slot], bytes);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (row[x] >= 0) {
              // chunk by chunk where the box is half a tile: a box lands its chunks one after another
              if (p.box == KT) {
                ptx::tma_load_4d(dst, map, &full[mine][slot], 0, off[x], row[x], 0);
              } else {
#pragma unroll 1
                for (int ch = 0; ch < D / 64; ++ch)
                  ptx::tma_load_4d(dst + ch * (KT * 128) + x * (p.box * 128), map, &full[mine][slot], 0, off[x], row[x], ch);
              }
            }
        } else {
          ptx::mbar_arrive(&full[mine][slot]);
        }
        ++g;
        if (!(g & 1) && g < groups) {
          cur.next(p);
          look_up();
        }
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      }
      idle = __any_sync(0xffffffffu, can) ? 0 : idle + 1;
      if (idle > p.wait_limit) *abort = 1;
      // a vote: a consumer may set the flag between two lanes' reads, and the
      // votes above need all lanes until all leave
      stop = __any_sync(0xffffffffu, *abort != 0);
    }
    // Each slot's newest copy lands before the CTA leaves, also where a consumer gives
    // up only after this (its copies are the ones that it no longer waits for).
    for (int x = g > NS ? g - NS : 0; x < g; ++x) ptx::mbar_wait_bounded(&full[mine][x % NS], (x / NS) & 1, kWaitPolls >> 6);
    __syncwarp();
  } else {
    // ---------------- consumers ----------------
    if (lane == 0) rec[warp] = Rec{};
    const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
    // place of 16-byte piece ch of row r in a slot
    auto piece = [](int r, int ch) { return static_cast<uint32_t>((ch >> 3) * (KT * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)); };
    // cp.async: K, V, K, V, ... of the part's tiles; the page ids are loaded a tile ahead
    Cursor<KT> ld = cur;
    TileRows<KT> rows;
    uint32_t row = ~0u;
    int issued = 0;
    if (!C::TMA && n > 0) rows.look_up(p, ld);
    auto issue = [&]() {
      if (C::TMA || issued >= 2 * n) return;
      const bool is_v = issued & 1;
      const int s = issued % NS;
      if (!is_v) {
        row = rows.row(p);
        const uint32_t mask = __ballot_sync(0xffffffffu, row != ~0u);
        if (lane == 0) live_mask[warp][s] = mask;
      }
      const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v : p.k);
      constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll
      for (int i = 0; i < KT * kChunks / 32; ++i) {
        const int x = i * 32 + lane, r = x / kChunks, ch = x % kChunks;
        const uint32_t pr = __shfl_sync(0xffffffffu, row, r);
        const int64_t at = (pr != ~0u ? static_cast<int64_t>(pr) * (D * 2) : 0) + ch * 16;
        cp_async_16(ring + s * C::kTile + piece(r, ch), src + at, pr != ~0u ? 16 : 0);  // no row: zeros
      }
      ++issued;
      if (is_v && issued < 2 * n) {
        ld.next(p);
        rows.look_up(p, ld);
      }
    };
    if (!C::TMA) {
      for (int s = 0; s < NS - 1; ++s) {
        issue();
        cp_async_commit();
      }
    }

    uint32_t qf[NT][D / 16][2];
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];
    static_assert(kRowsU * (kPad * 4 + 8) <= C::kRing, "a partial fits a warp's ring");
    int heads = 0;
    // (max in log2 units, sum) and the unnormalised rows of this warp's unit
    auto leave = [&](float2* ml, float* part, int stride) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int hr = nt * 8 + qi * 2 + h;
          if (hr < heads) {
            if (quad == 0) ml[hr] = make_float2(m[nt][h] * p.c, l[nt][h]);
            float* dst = part + hr * stride;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              dst[mt * 16 + quad] = o[mt][nt][h];
              dst[mt * 16 + 8 + quad] = o[mt][nt][h + 2];
            }
          }
        }
    };
    bool open = false;  // the unit's first tile of this warp's part has been taken
    int t_first = 0;
    int sk = 0, pk = 0;  // slot of the next tile, and its phase
    for (int it = 0; it < n; ++it) {
      if (!open) {
        open = true;
        t_first = cur.t;
        if (it == 0 && lane == 0) {
          rec[warp].n = n;
          rec[warp].b[0] = cur.b;
          rec[warp].u[0] = cur.u;
        }
        const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hr = gr * kRowsU + nt * 8 + quad;  // head within the KV head's group
          const int64_t q_at = cur.b * p.q_stride + static_cast<int64_t>(hk * p.g + hr) * D;
          const bool in = hr < p.g && q_in(p, q_at);
          const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + q_at);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            qf[nt][kk][0] = in ? qr[kk * 8 + qi] : 0u;
            qf[nt][kk][1] = in ? qr[kk * 8 + 4 + qi] : 0u;
          }
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }
      // K has landed
      if constexpr (C::TMA) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&full[warp][sk], pk, abort, p.wait_limit))) break;
      } else {
        cp_async_wait<NS - 2>();
        __syncwarp();  // for every lane, and V of the tile before has been read by every lane
      }
      const uint32_t mask = live_mask[warp][sk] & key_bits<KT>(cur.keys.lo, cur.keys.hi, cur.key0());
      if constexpr (!C::TMA) {
        issue();
        cp_async_commit();
      }
      const uint32_t ka = ring + sk * C::kTile;
      float sc[KS][NT][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[ks][nt][e] = 0.f;
        const int r = ks * 16 + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a0, a1, a2, a3;
          ptx::ldmatrix_x4(a0, a1, a2, a3, ka + piece(r, 2 * kk + (lane >> 4)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16_16816(sc[ks][nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
        }
      }
      if constexpr (C::TMA) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[warp][sk]);
      }
      if (++sk == NS) {
        sk = 0;
        pk ^= 1;
      }
      if (mask != kFull) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const bool k0 = (mask >> (ks * 16 + quad)) & 1, k1 = (mask >> (ks * 16 + 8 + quad)) & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (!k0) sc[ks][nt][0] = sc[ks][nt][1] = -INFINITY;
            if (!k1) sc[ks][nt][2] = sc[ks][nt][3] = -INFINITY;
          }
        }
      }
      float mn[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = -INFINITY;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) x = fmaxf(x, fmaxf(sc[ks][nt][h], sc[ks][nt][h + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mn[nt][h] = fmaxf(m[nt][h], x);
          grow |= mn[nt][h] > m[nt][h];
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float corr = m[nt][h] == -INFINITY ? 0.f : ptx::ex2((m[nt][h] - mn[nt][h]) * p.c);
            m[nt][h] = mn[nt][h];
            l[nt][h] *= corr;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              o[mt][nt][h] *= corr;
              o[mt][nt][h + 2] *= corr;
            }
          }
      }
      uint32_t pb[KS][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float mc0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] * p.c;
        const float mc1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] * p.c;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const float e0 = ptx::ex2(fmaf(sc[ks][nt][0], p.c, -mc0)), e1 = ptx::ex2(fmaf(sc[ks][nt][1], p.c, -mc1));
          const float e2 = ptx::ex2(fmaf(sc[ks][nt][2], p.c, -mc0)), e3 = ptx::ex2(fmaf(sc[ks][nt][3], p.c, -mc1));
          l[nt][0] += e0 + e2;
          l[nt][1] += e1 + e3;
          // P rounded to bf16 for the product (off by at most 2^-8 of each weight; the sum keeps fp32)
          pb[ks][nt][0] = ptx::movmatrix_trans(ptx::pack_bf16x2(e0, e1));
          pb[ks][nt][1] = ptx::movmatrix_trans(ptx::pack_bf16x2(e2, e3));
        }
      }
      // V has landed
      if constexpr (C::TMA) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&full[warp][sk], pk, abort, p.wait_limit))) break;
        if (mask != kFull) {
          // rows of masked keys, whatever they hold, become zeros: their P is 0, and 0 * NaN would be NaN
          uint8_t* vt = smem + warp * C::kRing + sk * C::kTile;
          for (int x = lane; x < KT * (D / 8); x += 32) {
            const int r = x / (D / 8);
            if (!((mask >> r) & 1)) *reinterpret_cast<uint4*>(vt + piece(r, x % (D / 8))) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();  // before the slot's next copy
          __syncwarp();
        }
      } else {
        cp_async_wait<NS - 2>();
        __syncwarp();  // for every lane, and K of this tile has been read by every lane
        issue();
        cp_async_commit();
      }
      const uint32_t va = ring + sk * C::kTile;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int r = ks * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          uint32_t a0, a1, a2, a3;
          ptx::ldmatrix_x4_trans(a0, a1, a2, a3, va + piece(r, 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16_16816(o[mt][nt], a0, a1, a2, a3, pb[ks][nt][0], pb[ks][nt][1]);
        }
      }
      if constexpr (C::TMA) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[warp][sk]);
      }
      if (++sk == NS) {
        sk = 0;
        pk ^= 1;
      }

      const bool unit_end = cur.t == cur.tiles - 1;
      if (unit_end || it == n - 1) {
        const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
        heads = min(kRowsU, p.g - gr * kRowsU);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
          }
        if (unit_end && t_first == 0) {
          const int64_t y_at = (static_cast<int64_t>(cur.b) * p.Hq + hk * p.g + gr * kRowsU) * D;
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + y_at;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float i0 = l[nt][0] != 0.f ? 1.f / l[nt][0] : 0.f, i1 = l[nt][1] != 0.f ? 1.f / l[nt][1] : 0.f;
            const int hr = nt * 8 + quad;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              const uint32_t x = ptx::movmatrix_trans(ptx::pack_bf16x2(o[mt][nt][0] * i0, o[mt][nt][1] * i1));
              const uint32_t z = ptx::movmatrix_trans(ptx::pack_bf16x2(o[mt][nt][2] * i0, o[mt][nt][3] * i1));
              if (hr < heads && y_in(p, y_at + hr * D + mt * 16, 16)) {
                uint32_t* yr = reinterpret_cast<uint32_t*>(y + hr * D + mt * 16);
                yr[qi] = x;
                yr[4 + qi] = z;
              }
            }
          }
        } else if (it < n - 1) {
          // the first unit of the part, begun before it: to the workspace, the ring is still streaming
          const int64_t at = (static_cast<int64_t>(cta) * W + warp) * kRowsU;
          if (part_in(p, at, heads, static_cast<int64_t>(p.slices) * W)) leave(p.w_ml + at, p.w_part + at * D, D);
          if (lane == 0) rec[warp].early = 1;
        } else {
          // the last unit of the part: into the ring, which has been read
          if (!C::TMA) cp_async_wait<0>();
          __syncwarp();
          float* dst = reinterpret_cast<float*>(smem + warp * C::kRing);
          leave(reinterpret_cast<float2*>(dst + kRowsU * kPad), dst, kPad);
          if (lane == 0) {
            rec[warp].late = 1;
            rec[warp].begins = t_first == 0;
            rec[warp].ends = unit_end;
            rec[warp].b[1] = cur.b;
            rec[warp].u[1] = cur.u;
          }
        }
        open = false;
      }
      cur.next(p);
    }
  }

  // ---- the units split over this CTA's warps (and maybe its neighbours)
  __syncthreads();
  const bool dead = C::TMA && *abort;  // nothing to join: a part is missing
  if (dead && tid == 0) report(p.status, EXTKV_DEV_TIMEOUT);
  if (!C::CLUSTER && dead) return;
  float* share = reinterpret_cast<float*>(smem + W * C::kRing);  // cluster: this CTA's rows, then their (max, sum)
  float2* share_ml = reinterpret_cast<float2*>(share + kRowsU * D);
  if (warp == 0) {
    // lane k looks at warp k's part; a unit's warps are neighbours, so the
    // members of a chain are the late partials of its unit and the early one
    // that ends it, if there is one
    const Rec r = rec[min(lane, W - 1)];
    const bool some = lane < W && r.n > 0;
    const unsigned busy = __ballot_sync(0xffffffffu, some);
    const int64_t head = static_cast<int64_t>(r.b[0]) * p.units + r.u[0];
    const int64_t last = static_cast<int64_t>(r.b[1]) * p.units + r.u[1];
    const unsigned behind = busy & (lane < 31 ? ~0u << (lane + 1) : 0u);
    const int64_t next_head = __shfl_sync(0xffffffffu, head, behind ? __ffs(behind) - 1 : 0);
    const bool late = some && r.late, early = some && r.early;
    const bool ends_late = late && !(behind && next_head == last);
    const int64_t first = __shfl_sync(0xffffffffu, head, busy ? __ffs(busy) - 1 : 0);
    int c = 0;
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {  // 0: ended by w's early partial, 1: by its late one
        if (!__shfl_sync(0xffffffffu, kind ? ends_late : early, w)) continue;
        const int64_t id = __shfl_sync(0xffffffffu, kind ? last : head, w);
        const unsigned members = __ballot_sync(0xffffffffu, late && last == id);
        const int k0 = members ? __ffs(members) - 1 : 0;
        const bool begins = __shfl_sync(0xffffffffu, r.begins, k0) && members;
        const bool ends = kind ? __shfl_sync(0xffffffffu, r.ends, w) : true;
        if (lane == 0) {
          Chain x;
          x.members = members;
          x.early = kind ? -1 : w;
          x.b = static_cast<int>(id / p.units);
          x.u = static_cast<int>(id - static_cast<int64_t>(x.b) * p.units);
          x.whole = begins && ends;
          x.slot = id == first ? 0 : 1;  // where the merge kernel looks: the CTA's first unit, or its last
          chains[c] = x;
        }
        ++c;
      }
    if (lane == 0) n_chains = c;
  }
  __syncthreads();
  for (int c = 0; c < n_chains; ++c) {
    const Chain x = chains[c];
    const int hk = x.u / p.groups, gr = x.u - hk * p.groups, heads = min(kRowsU, p.g - gr * kRowsU);
    for (int i = tid; i < heads * (D / 4); i += C::kThreads) {
      const int r = i / (D / 4), c4 = i - r * (D / 4);
      // the members' (max, sum) and four columns of their rows, all in flight at once
      float2 ml[W + 1];
      float4 v[W + 1];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float* src = reinterpret_cast<const float*>(smem + k * C::kRing);
        const bool in = (x.members >> k) & 1;
        ml[k] = in ? reinterpret_cast<const float2*>(src + kRowsU * kPad)[r] : make_float2(-INFINITY, 0.f);
        v[k] = in ? reinterpret_cast<const float4*>(src + r * kPad)[c4] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      ml[W] = make_float2(-INFINITY, 0.f);
      v[W] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x.early >= 0) {
        const int64_t at = (static_cast<int64_t>(cta) * W + x.early) * kRowsU + r;
        if (part_in(p, at, 1, static_cast<int64_t>(p.slices) * W)) {
          ml[W] = __ldcg(p.w_ml + at);
          v[W] = __ldcg(reinterpret_cast<const float4*>(p.w_part + at * D) + c4);
        }
      }
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k <= W; ++k) M = fmaxf(M, ml[k].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k <= W; ++k) {
        const float wt = ml[k].x == -INFINITY ? 0.f : ptx::ex2(ml[k].x - ref);  // -inf: absent, or every key skipped
        L = fmaf(wt, ml[k].y, L);
        acc.x = fmaf(wt, v[k].x, acc.x);
        acc.y = fmaf(wt, v[k].y, acc.y);
        acc.z = fmaf(wt, v[k].z, acc.z);
        acc.w = fmaf(wt, v[k].w, acc.w);
      }
      if (x.whole) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        const int64_t y_at = (static_cast<int64_t>(x.b) * p.Hq + hk * p.g + gr * kRowsU + r) * D;
        uint2* y = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + y_at);
        if (y_in(p, y_at + 4 * c4, 4))
          y[c4] = make_uint2(ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
      } else if constexpr (C::CLUSTER) {
        if (c4 == 0) share_ml[r] = make_float2(M, L);
        reinterpret_cast<float4*>(share + r * D)[c4] = acc;
      } else {
        const int64_t at = (static_cast<int64_t>(cta) * 2 + x.slot) * kRowsU + r;
        if (part_in(p, at, 1, static_cast<int64_t>(p.slices) * 2)) {
          if (c4 == 0) p.ml[at] = make_float2(M, L);
          reinterpret_cast<float4*>(p.part + at * D)[c4] = acc;
        }
      }
    }
  }
  if constexpr (C::CLUSTER) {
    const int unit = cta / p.cluster, b = unit / p.units, u = unit - b * p.units;
    const int hk = u / p.groups, gr = u - hk * p.groups, heads = min(kRowsU, p.g - gr * kRowsU);
    if (tiles_here == 0 && tid < kRowsU) share_ml[tid] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    ptx::cluster_sync();
    const int64_t y_at = (static_cast<int64_t>(b) * p.Hq + hk * p.g + gr * kRowsU) * D;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + y_at;
    if (unit_tiles != 1 && !dead) {  // one tile: a warp has written the rows
      for (int i = rank * C::kThreads + tid; i < heads * (D / 4); i += p.cluster * C::kThreads) {
        const int r = i / (D / 4), c4 = i - r * (D / 4);
        float2 ml[kMaxCluster];
        float4 v[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          ml[k] = make_float2(-INFINITY, 0.f);
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < p.cluster) {
            const uint32_t at = ptx::map_cluster(share_ml + r, k);
            ml[k] = make_float2(ptx::ld_cluster_f32(at), ptx::ld_cluster_f32(at + 4));
            if (!(ml[k].x == -INFINITY && ml[k].y == 0.f)) v[k] = ptx::ld_cluster_f32x4(ptx::map_cluster(share + r * D + 4 * c4, k));
          }
        }
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, ml[k].x);
        const float ref = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          const float wt = ml[k].x == -INFINITY ? 0.f : ptx::ex2(ml[k].x - ref);
          L = fmaf(wt, ml[k].y, L);
          acc.x = fmaf(wt, v[k].x, acc.x);
          acc.y = fmaf(wt, v[k].y, acc.y);
          acc.z = fmaf(wt, v[k].z, acc.z);
          acc.w = fmaf(wt, v[k].w, acc.w);
        }
        const float inv = L != 0.f ? 1.f / L : 0.f;  // no key: a zero row
        if (y_in(p, y_at + static_cast<int64_t>(r) * D + 4 * c4, 4))
          reinterpret_cast<uint2*>(y + static_cast<int64_t>(r) * D)[c4] =
              make_uint2(ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
      }
    }
    __syncwarp();
    ptx::cluster_sync();  // a CTA's share stays until its peers have read it
  }
}

// ---- SIMT (fp32, other head sizes) ---------------------------------------------------

constexpr int kSimtWarps = 3;
constexpr int kSimtStages = 2;

// Row stride in shared memory: 16 bytes of padding, so that the keys' rows
// start in different banks.
template <typename T>
__host__ __device__ constexpr int simt_stride(int D) {
  return D + 16 / static_cast<int>(sizeof(T));
}

template <typename T, int DPL, int KT>
__global__ void __launch_bounds__(kSimtWarps * 32, 1) paged_decode_simt_kernel(const PagedParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t pre[kSimtWarps * 32 + 1], warp_sum[kSimtWarps];
  __shared__ uint32_t live_mask[kSimtWarps][kSimtStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.D;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const bool few = p.B <= 32;
  const LaneScan<KT> scan(p);
  int per = 0;
  if (!few) per = scan_tiles<KT>(p, pre, warp_sum);
  const Axis axis(p, few ? scan.total(p) : pre[blockDim.x] * p.units);
  const int slice = warp * gridDim.x + blockIdx.x;  // few tiles: one warp per SM first
  if (slice >= axis.n) return;
  const int64_t f0 = axis.start(slice), f1 = axis.start(slice + 1);
  const int n = static_cast<int>(f1 - f0);  // at least one

  const int stride = simt_stride<T>(D);
  const int stage = 2 * KT * stride;  // elements
  const int q_bytes = (kRows * D + kRows * KT) * 4;
  uint8_t* mine = smem + warp * (kSimtStages * stage * static_cast<int>(sizeof(T)) + q_bytes);
  T* ring = reinterpret_cast<T*>(mine);
  float* qs = reinterpret_cast<float*>(mine + kSimtStages * stage * sizeof(T));
  float* ps = qs + kRows * D;
  const int chunks = D * static_cast<int>(sizeof(T)) / 16;
  const int row_bytes = D * static_cast<int>(sizeof(T));

  Cursor<KT> ld = few ? scan.cursor_at(p, f0) : cursor_at<KT>(p, pre, per, f0);
  Cursor<KT> cur = ld;
  TileRows<KT> rows;
  rows.look_up(p, ld);
  int issued = 0;
  auto issue = [&]() {
    const int s = issued % kSimtStages;
    const uint32_t row = rows.row(p);
    const uint32_t mask = __ballot_sync(0xffffffffu, row != ~0u);
    if (lane == 0) live_mask[warp][s] = mask;
    const uint32_t kd = ptx::smem_u32(ring + s * stage), vd = kd + KT * stride * sizeof(T);
    for (int i = 0; i < KT * chunks; i += 32) {  // whole warps: the shuffle is read by every lane
      const int x = i + lane, r = min(x / chunks, KT - 1), ch = x - r * chunks;
      const uint32_t pr = __shfl_sync(0xffffffffu, row, r);
      if (x < KT * chunks) {
        const uint32_t bytes = pr != ~0u ? 16 : 0;
        const int64_t at = (pr != ~0u ? static_cast<int64_t>(pr) * row_bytes : 0) + ch * 16;
        const uint32_t to = r * stride * sizeof(T) + ch * 16;
        cp_async_16(kd + to, static_cast<const uint8_t*>(p.k) + at, bytes);
        cp_async_16(vd + to, static_cast<const uint8_t*>(p.v) + at, bytes);
      }
    }
    ++issued;
    if (issued < n) {
      ld.next(p);
      rows.look_up(p, ld);
    }
  };
  issue();
  cp_async_commit();

  SimtState<DPL> st;
  st.clear();
  bool open = false;
  int t_first = 0, slot = 0;
  for (int it = 0; it < n; ++it) {
    const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
    const int heads = min(kRows, p.g - gr * kRows);
    if (!open) {
      open = true;
      t_first = cur.t;
      st.clear();
      const int64_t q_at = cur.b * p.q_stride + static_cast<int64_t>(hk * p.g + gr * kRows) * D;
      const T* q = static_cast<const T*>(p.q) + q_at;
      simt_stage_q<T, DPL>(qs, D, p.c, [&](int r) {
        return r < heads && q_in(p, q_at + static_cast<int64_t>(r) * D) ? q + static_cast<int64_t>(r) * D : nullptr;
      });
    }
    __syncwarp();  // tile it - 1 has been read by every lane
    if (issued < n) issue();
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const int s = it % kSimtStages;
    const uint32_t mask = live_mask[warp][s];
    const T* kt = ring + s * stage;
    // live keys of a tile: whole runs, as pages end; a bad page inside a tile
    // leaves a gap, taken run by run
    uint32_t left = mask;
    while (left) {
      const int a = __ffs(left) - 1;
      const uint32_t run = ~(left >> a);
      const int b = run ? min(32, a + __ffs(run) - 1) : 32;
      int lo[kRows], hi[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        lo[r] = a;
        hi[r] = b;
      }
      simt_tile<T, DPL, KT>(st, kt, kt + KT * stride, stride, qs, ps, D, lo, hi);
      left = b >= 32 ? 0u : left & (~0u << b);
    }

    const bool unit_end = cur.t == cur.tiles - 1;
    if (unit_end || it == n - 1) {
      const bool whole = unit_end && t_first == 0;
      st.reduce();
      const int64_t y_at = (static_cast<int64_t>(cur.b) * p.Hq + hk * p.g + gr * kRows) * D;
      T* y = static_cast<T*>(p.y) + y_at;
      const int64_t at = (static_cast<int64_t>(slice) * 2 + slot) * kRows;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r < heads && (whole ? y_in(p, y_at + r * D, D) : part_in(p, at + r, 1, static_cast<int64_t>(p.slices) * 2))) {
          const float inv = st.l[r] != 0.f ? 1.f / st.l[r] : 0.f;
          if (!whole && lane == 0) p.ml[at + r] = make_float2(st.m[r], st.l[r]);
#pragma unroll
          for (int i = 0; i < DPL; ++i) {
            const int d = lane + 32 * i;
            if (d < D) {
              if (whole) y[r * D + d] = Elem<T>::from_float(st.acc[r][i] * inv);
              else p.part[(at + r) * D + d] = st.acc[r][i];
            }
          }
        }
      }
      slot = 1;
      open = false;
    }
    cur.next(p);
  }
}

// ---- joining the units split over slices -----------------------------------------------

// One CTA per (sequence, query head).  A unit's partials lie in the slices that
// hold its tiles: the first of them may have ended an earlier unit before it
// (then its partial is in the second place), the others begin with it.  The
// slices' weights exp2(max_s - M) go to shared memory; then a thread owns four
// columns and every kSub-th slice, eight loads in flight, and the kSub sums are
// added in order.
constexpr int kMergeThreads = 256;
constexpr int kMaxSlices = 2048;

template <typename T>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedParams p) {
  __shared__ float w_s[kMaxSlices];
  __shared__ float4 acc_s[kMergeThreads];
  __shared__ float red[2][kMergeThreads / 32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.Hq, h = blockIdx.x - b * p.Hq, D = p.D;
  const int hk = h / p.g, hr = h - hk * p.g, gr = hr / p.rows, r = hr - gr * p.rows;
  if (!(base_in(p, b) && base_in(p, b + 1))) return;
  const int64_t b0 = p.base[b], tiles = p.base[b + 1] - b0, total = p.base[p.B] * p.units;
  const int64_t y_at = (static_cast<int64_t>(b) * p.Hq + h) * D;
  T* y = static_cast<T*>(p.y) + y_at;
  if (!y_in(p, y_at, D)) return;
  if (tiles == 0) {  // no key
    for (int d = tid; d < D; d += kMergeThreads) y[d] = Elem<T>::from_float(0.f);
    return;
  }
  const Axis axis(p, total);
  const int64_t u0 = b0 * p.units + static_cast<int64_t>(hk * p.groups + gr) * tiles;
  const int s0 = axis.holds(u0), s1 = axis.holds(u0 + tiles - 1);
  if (s0 == s1) return;  // written by the slice itself
  const int first_slot = axis.start(s0) < u0 ? 1 : 0;
  const int n = s1 - s0 + 1;
  // partial i of the unit, in rows of the workspace
  auto at = [&](int i) { return (static_cast<int64_t>(s0 + i) * 2 + (i == 0 ? first_slot : 0)) * p.rows + r; };
  auto there = [&](int i) { return part_in(p, at(i), 1, static_cast<int64_t>(p.slices) * 2); };

  // four columns of the first partials this thread adds up: on their way while
  // the weights are computed
  const int cols = D / 4, subs = kMergeThreads / cols;  // D <= 512: two at least
  const int sub = tid / cols, c = tid - sub * cols;
  const float4* part = reinterpret_cast<const float4*>(p.part) + c;
  constexpr int kAhead = 8;
  float4 v[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * subs;
      v[u] = sub < subs && i < n && there(i) ? __ldcg(part + at(i) * cols) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  fetch(sub);

  float M = -INFINITY;
  for (int i = tid; i < n; i += kMergeThreads) {
    const float m = there(i) ? __ldcg(&p.ml[at(i)].x) : -INFINITY;
    w_s[i] = m;
    M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) M = fmaxf(M, red[0][i]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int i = tid; i < n; i += kMergeThreads) {
    const float w = w_s[i] == -INFINITY ? 0.f : ptx::ex2(w_s[i] - ref);  // -inf: every key of the slice was skipped
    w_s[i] = w;
    if (there(i)) L = fmaf(w, __ldcg(&p.ml[at(i)].y), L);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) L += red[1][i];

  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = sub; i0 < n; i0 += kAhead * subs) {
    if (i0 != sub) fetch(i0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * subs;
      const float w = i < n ? w_s[i] : 0.f;
      a.x = fmaf(w, v[u].x, a.x);
      a.y = fmaf(w, v[u].y, a.y);
      a.z = fmaf(w, v[u].z, a.z);
      a.w = fmaf(w, v[u].w, a.w);
    }
  }
  if (sub < subs) acc_s[tid] = a;
  __syncthreads();
  if (sub == 0) {
    for (int u = 1; u < subs; ++u) {
      const float4 v = acc_s[u * cols + c];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    T* yc = y + 4 * c;
    yc[0] = Elem<T>::from_float(a.x * inv);
    yc[1] = Elem<T>::from_float(a.y * inv);
    yc[2] = Elem<T>::from_float(a.z * inv);
    yc[3] = Elem<T>::from_float(a.w * inv);
  }
}

// ---- host ------------------------------------------------------------------------------

struct Plan {
  int rows, groups, warps, slices;
  size_t off_ml, off_part, off_w_ml, off_w_part, bytes;
};

bool use_mma(int64_t D, int dtype) {
  return dtype == EXTKV_BF16 && (D == 64 || D == 128 || D == 256 || D == 512);
}

// Sixteen heads a unit where the KV head has more than eight and their
// accumulators fit the registers (D/4 a thread and eight heads).
int unit_rows(int64_t g, int64_t D, bool mma) { return mma && g > 8 && D <= 256 ? 16 : 8; }

// Consumer warps of the tensor-core kernels.
int mma_warps(int64_t D) { return D == 256 ? 4 : 6; }

Plan plan_of(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  const bool mma = use_mma(D, dtype);
  Plan pl;
  const int64_t g = Hq / Hkv;
  pl.rows = unit_rows(g, D, mma);
  pl.groups = static_cast<int>((g + pl.rows - 1) / pl.rows);
  pl.warps = mma ? mma_warps(D) : kSimtWarps;
  pl.slices = mma ? std::min(num_sms(), kMaxSlices) : std::min(num_sms() * pl.warps, kMaxSlices / pl.warps * pl.warps);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  pl.off_ml = up(sizeof(int64_t) * (B + 1));
  pl.off_part = pl.off_ml + up(sizeof(float2) * 2 * pl.slices * pl.rows);
  pl.off_w_ml = pl.off_part + up(sizeof(float) * 2 * pl.slices * pl.rows * D);
  pl.off_w_part = pl.off_w_ml + (mma ? up(sizeof(float2) * pl.slices * pl.warps * pl.rows) : 0);
  pl.bytes = pl.off_w_part + (mma ? up(sizeof(float) * pl.slices * pl.warps * pl.rows * D) : 0);
  return pl;
}

// The launch configuration of a cluster kernel.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ClusterLaunch(int clusters, int size, int threads, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters) * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// Clusters of `size` CTAs that can run at once, per kernel and device.  (One
// sixteenth off: the query has been seen to count clusters that the hardware
// then placed one after another.)
int clusters_at_once(const void* kernel, int size, int threads, size_t smem) {
  struct Entry {
    const void* kernel;
    int dev, size, n;
  };
  static std::mutex mu;
  static Entry entries[64];
  static int used = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> g(mu);
  for (int i = 0; i < used; ++i)
    if (entries[i].kernel == kernel && entries[i].dev == dev && entries[i].size == size) return entries[i].n;
  int n = 0;
  if (set_max_dynamic_smem(kernel, smem) == cudaSuccess) {
    ClusterLaunch l(1, size, threads, smem, nullptr);
    l.cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg) != cudaSuccess) n = 0;
    n -= (n + 15) / 16;
  }
  (void)cudaGetLastError();
  if (used < 64) entries[used++] = Entry{kernel, dev, size, n};
  return n;
}

// CTAs per unit on the cluster kernel, or 0: the axis of tiles.  A cluster's time
// follows its unit's longest share, bounded by the window or the table's
// capacity; the axis' follows the average, plus about 4 us of joining CTAs, in
// which an SM streams some 180 KB.  Measured (axis, cluster): 1 sequence of 517,
// 8 KV heads of 256: 12.2, 9.7 us; 8 sequences of 8, window 1024: 22.5, 20.2 us.
// The lengths are on the device, so without a window the bound is the table's
// width: that one sequence in a table of 8192 slots runs on the axis (2.7 us more).
template <class C>
int cluster_size(const PagedParams& p, bool forced) {
  const int64_t units = static_cast<int64_t>(p.B) * p.units;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t in_window = static_cast<int64_t>(p.window) + C::KT;  // windows go up to 2^31 - 1
  const int64_t keys = p.window > 0 && in_window < cap ? in_window : cap;
  const double longest = static_cast<double>(keys) * C::D * 4;  // bytes of a unit
  const void* k = reinterpret_cast<const void*>(paged_decode_mma_kernel<C>);
  for (int c = kMaxCluster; c > 1; c /= 2) {
    if (!forced && longest * (1.0 / c - static_cast<double>(units) / num_sms()) > 180e3) continue;
    if (units <= clusters_at_once(k, c, C::kThreads, C::kSmem)) return c;
  }
  return 0;
}

template <class C>
cudaError_t launch_mma_cfg(PagedParams p, cudaStream_t s) {
  auto k = paged_decode_mma_kernel<C>;
  CUtensorMap kmap, vmap;
  std::memset(&kmap, 0, sizeof kmap);
  std::memset(&vmap, 0, sizeof vmap);
  if (C::TMA) {
    // (64 columns, row of a page, page and head, 64-column chunk)
    p.box = p.page_size % C::KT == 0 ? C::KT : 16;
    const uint64_t dims[4] = {64, static_cast<uint64_t>(p.page_size), static_cast<uint64_t>(p.num_pages) * p.Hkv, C::D / 64};
    const uint64_t str[3] = {C::D * 2, static_cast<uint64_t>(p.page_size) * C::D * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(p.box), 1, p.box == C::KT ? C::D / 64u : 1u};
    if (!make_tensor_map_bf16(&kmap, p.k, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_bf16(&vmap, p.v, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), C::kSmem); e != cudaSuccess) return e;
  cudaError_t e;
  if constexpr (C::CLUSTER) {
    ClusterLaunch l(p.B * p.units, p.cluster, C::kThreads, C::kSmem, s);
    e = cudaLaunchKernelEx(&l.cfg, k, kmap, vmap, p);
  } else {
    PdlLaunch l(dim3(p.slices), C::kThreads, C::kSmem, s);
    e = cudaLaunchKernelEx(&l.cfg, k, kmap, vmap, p);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

// p.cluster: 0 where the merge kernel has to follow
template <int D, int NT, int KT, int SLOTS, int WARPS>
cudaError_t launch_mma(PagedParams& p, int variant, cudaStream_t s) {
  // A request is a box of 16 rows at least: pages of other sizes take cp.async.
  // (The strides of a tensor map end at 2^40 bytes.)
  const bool tma = p.page_size % 16 == 0 && static_cast<int64_t>(p.page_size) * D * 2 < (int64_t(1) << 40);
  if (variant == kDecodeCluster && !tma) return cudaErrorNotSupported;
  if (!tma) return launch_mma_cfg<MmaCfg<D, NT, KT, SLOTS, WARPS, false>>(p, s);
  if (variant != kDecodeStreamK)
    p.cluster = cluster_size<MmaCfg<D, NT, KT, SLOTS, WARPS, true, true>>(p, variant == kDecodeCluster);
  if (variant == kDecodeCluster && !p.cluster) return cudaErrorNotSupported;
  return p.cluster ? launch_mma_cfg<MmaCfg<D, NT, KT, SLOTS, WARPS, true, true>>(p, s)
                   : launch_mma_cfg<MmaCfg<D, NT, KT, SLOTS, WARPS, true>>(p, s);
}

template <typename T, int DPL, int KT>
cudaError_t launch_simt(const PagedParams& p, cudaStream_t s) {
  const size_t smem = kSimtWarps * (kSimtStages * 2 * KT * simt_stride<T>(p.D) * sizeof(T) +
                                    static_cast<size_t>(kRows * p.D + kRows * KT) * 4);
  auto k = paged_decode_simt_kernel<T, DPL, KT>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), smem); e != cudaSuccess) return e;
  PdlLaunch l(dim3(p.slices / kSimtWarps), kSimtWarps * 32, smem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_d(const PagedParams& p, cudaStream_t s) {
  if (p.D <= 64) return launch_simt<T, 2, 32>(p, s);
  if (p.D <= 128) return launch_simt<T, 4, 32>(p, s);
  if (p.D <= 256) return launch_simt<T, 8, 16>(p, s);
  return launch_simt<T, 16, 4>(p, s);  // 148 KB of shared memory in fp32
}

template <typename T>
cudaError_t launch_merge(const PagedParams& p, cudaStream_t s) {
  PdlLaunch l(dim3(static_cast<unsigned>(p.B * p.Hq)), kMergeThreads, 0, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, paged_merge_kernel<T>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t paged_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  return plan_of(B, Hq, Hkv, D, dtype).bytes;
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, const char** name) {
  const Plan pl = plan_of(a.B, a.Hq, a.Hkv, a.D, a.dtype);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PagedParams p{};
  p.y = a.y;
  p.q = a.q;
  p.k = a.k_pages;
  p.v = a.v_pages;
  p.table = a.page_table;
  p.nonpad = a.nonpad;
  p.c = a.scale * kLog2e;
  p.window = a.window > 0 ? a.window : 0;
  p.B = static_cast<int>(a.B);
  p.Hq = static_cast<int>(a.Hq);
  p.Hkv = static_cast<int>(a.Hkv);
  p.g = p.Hq / p.Hkv;
  p.D = static_cast<int>(a.D);
  p.page_size = static_cast<int>(a.page_size);
  p.max_pages = static_cast<int>(a.max_pages);
  p.num_pages = a.num_pages;
  p.q_stride = a.q_stride;
  p.rows = pl.rows;
  p.groups = pl.groups;
  p.units = pl.groups * p.Hkv;
  p.slices = pl.slices;
  p.base = reinterpret_cast<int64_t*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  p.part = reinterpret_cast<float*>(ws + pl.off_part);
  p.w_ml = reinterpret_cast<float2*>(ws + pl.off_w_ml);
  p.w_part = reinterpret_cast<float*>(ws + pl.off_w_part);
  p.status = a.status;
  p.wait_limit = wait_limit(a.wait_limit_plus1, kWaitPolls);
  cudaError_t e;
  if (use_mma(a.D, a.dtype)) {
    *name = "paged_decode_mma";
    const bool two = pl.rows == 16;
    if (a.D == 64) e = two ? launch_mma<64, 2, 32, 8, 6>(p, a.variant, a.stream) : launch_mma<64, 1, 32, 8, 6>(p, a.variant, a.stream);
    else if (a.D == 128) e = two ? launch_mma<128, 2, 32, 4, 6>(p, a.variant, a.stream) : launch_mma<128, 1, 32, 4, 6>(p, a.variant, a.stream);
    else if (a.D == 256) e = two ? launch_mma<256, 2, 16, 6, 4>(p, a.variant, a.stream) : launch_mma<256, 1, 16, 6, 4>(p, a.variant, a.stream);
    else e = launch_mma<512, 1, 16, 2, 6>(p, a.variant, a.stream);
  } else {
    if (a.variant == kDecodeCluster) return cudaErrorNotSupported;
    *name = a.dtype == EXTKV_F32 ? "paged_decode_simt_f32" : "paged_decode_simt_bf16";
    e = a.dtype == EXTKV_F32 ? launch_simt_d<float>(p, a.stream) : launch_simt_d<__nv_bfloat16>(p, a.stream);
  }
  if (e != cudaSuccess) return e;
  if (p.cluster) {
    *name = "paged_decode_cluster";
    note_launches(1);
    return cudaSuccess;
  }
  e = a.dtype == EXTKV_F32 ? launch_merge<float>(p, a.stream) : launch_merge<__nv_bfloat16>(p, a.stream);
  if (e == cudaSuccess) note_launches(2);
  return e;
}

}  // namespace extkv
