// paged_decode.cu -- attention of one new token per sequence over a cache in
// pages.
//
// Bound: HBM.  Every live K and V row is read once per KV head (4 D bytes for
// bf16), for 4 D (Hq/Hkv) flops.
//
// The batch's work is one axis of tiles (KT keys of one unit; a unit is a
// (sequence, KV head, group of query heads)), unit after unit, and every warp
// of the GPU takes an equal contiguous slice of it, whatever the sequences'
// lengths are: a warp streams its slice through its own ring of shared-memory
// stages (16-byte cp.async, a row's address from the page table, rows outside
// the sequence filled with zeros), so warps never wait for each other and a
// page may end anywhere in a tile.  A unit that lies in one slice is written
// out by its warp; of a unit split over slices each warp leaves (max, sum,
// unnormalised output) in the workspace, and the merge kernel joins them in
// slice order, so the result does not depend on timing.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "simt_tile.cuh"
#include "tma_host.h"

namespace extkv {

namespace {

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
  int rows;    // query heads per unit (the kernel's row capacity)
  int groups;  // units per (sequence, KV head)
  int units;   // groups * Hkv: units of a sequence
  int slices;
  int64_t* base;  // [B + 1] tiles before each sequence (per unit of it)
  float2* ml;     // [slices][2][rows] (max in log2 units, sum)
  float* part;    // [slices][2][rows][D]
  int32_t* status;
};

struct LiveKeys {
  int lo, hi;
};

__device__ __forceinline__ LiveKeys live_keys(const PagedParams& p, int b) {
  const int64_t np = p.nonpad[b];
  if (np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size) return {0, 0};
  const int n = static_cast<int>(np);
  return {p.window > 0 && n > p.window ? n - p.window : 0, n};
}

template <int KT>
__device__ __forceinline__ int tiles_of(LiveKeys k) {
  return (k.hi - k.lo + KT - 1) / KT;
}

// Slices the axis is cut into: one per warp, or one per tile when there are fewer.
__device__ __forceinline__ int live_slices(const PagedParams& p, int64_t total) {
  return total < p.slices ? static_cast<int>(total) : p.slices;
}

// A position on the axis of tiles.
template <int KT>
struct Cursor {
  int b, u, t, tiles;
  LiveKeys keys;
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
      p.base[b] = at;
      at += tiles_of<KT>(live_keys(p, b));
      const int64_t np = p.nonpad[b];
      if (np < 0 || np > static_cast<int64_t>(p.max_pages) * p.page_size) report(p.status, EXTKV_DEV_BAD_NONPAD);
    }
    if (tid == nt - 1) p.base[p.B] = pre[nt];
  }
  return per;
}

// The cursor at tile f of the axis (f < total).
template <int KT>
__device__ __forceinline__ Cursor<KT> cursor_at(const PagedParams& p, const int64_t* pre, int per, int64_t f) {
  int lo = 0, hi = blockDim.x;  // the last chunk whose first tile is <= f
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * p.units <= f) lo = mid;
    else hi = mid;
  }
  int64_t rest = f - pre[lo] * p.units;
  Cursor<KT> c;
  c.b = lo * per;
  for (;;) {
    c.keys = live_keys(p, c.b);
    c.tiles = tiles_of<KT>(c.keys);
    const int64_t n = static_cast<int64_t>(c.tiles) * p.units;
    if (rest < n) break;
    rest -= n;
    ++c.b;
  }
  c.u = static_cast<int>(rest / c.tiles);
  c.t = static_cast<int>(rest - static_cast<int64_t>(c.u) * c.tiles);
  return c;
}

// Pool rows of a tile, one per lane: the page id is loaded a tile ahead.
template <int KT>
struct TileRows {
  int64_t page;
  int off, u;
  bool live;
  __device__ __forceinline__ void look_up(const PagedParams& p, const Cursor<KT>& c) {
    const int lane = threadIdx.x & 31;
    const int j = c.keys.lo + c.t * KT + lane;
    live = lane < KT && j < c.keys.hi;
    u = c.u;
    off = 0;
    page = -1;
    if (live) {
      const int pg = j / p.page_size;
      off = j - pg * p.page_size;
      page = p.table[static_cast<int64_t>(c.b) * p.max_pages + pg];
    }
  }
  // row of the pool in units of D elements, or ~0
  __device__ __forceinline__ uint32_t row(const PagedParams& p) const {
    if (!live) return ~0u;
    if (page < 0 || page >= p.num_pages) {
      if (u == 0 && ((threadIdx.x & 31) == 0 || off == 0)) report(p.status, EXTKV_DEV_BAD_PAGE);
      return ~0u;
    }
    const int64_t r = (page * p.Hkv + u / p.groups) * p.page_size + off;
    if (!EXTKV_IN(r, 1, p.num_pages * p.Hkv * p.page_size, p.status)) return ~0u;
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

template <int D_, int NT_, int KT_, int STAGES_, int WARPS_>
struct MmaCfg {
  static constexpr int D = D_, NT = NT_, KT = KT_, STAGES = STAGES_, WARPS = WARPS_;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTile = KT * kRowBytes;  // one of K, V
  static constexpr int kStage = 2 * kTile;
  static constexpr int kSmem = WARPS * STAGES * kStage;
};

template <class C>
__global__ void __launch_bounds__(C::WARPS * 32, 1) paged_decode_mma_kernel(const PagedParams p) {
  constexpr int D = C::D, NT = C::NT, KT = C::KT, ST = C::STAGES, KS = KT / 16;
  constexpr int kRowsU = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t pre[C::WARPS * 32 + 1], warp_sum[C::WARPS];
  __shared__ uint32_t live_mask[C::WARPS][ST];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane >> 2, qi = lane & 3;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int per = scan_tiles<KT>(p, pre, warp_sum);
  const int64_t total = pre[blockDim.x] * p.units;
  const int slice = warp * gridDim.x + blockIdx.x;  // few tiles: one warp per SM first
  const int slices = live_slices(p, total);
  if (slice >= slices) return;
  const int64_t f0 = total * slice / slices, f1 = total * (slice + 1) / slices;
  const int n = static_cast<int>(f1 - f0);  // at least one

  const uint32_t ring = ptx::smem_u32(smem) + warp * ST * C::kStage;
  Cursor<KT> ld = cursor_at<KT>(p, pre, per, f0);
  Cursor<KT> cur = ld;
  TileRows<KT> rows;
  rows.look_up(p, ld);
  const uint8_t* kp = static_cast<const uint8_t*>(p.k);
  const uint8_t* vp = static_cast<const uint8_t*>(p.v);

  int issued = 0;
  auto issue = [&]() {
    const int s = issued % ST;
    const uint32_t row = rows.row(p);
    const uint32_t mask = __ballot_sync(0xffffffffu, row != ~0u);
    if (lane == 0) live_mask[warp][s] = mask;
    const uint32_t kd = ring + s * C::kStage, vd = kd + C::kTile;
    constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < KT * kChunks / 32; ++i) {
      const int x = i * 32 + lane, r = x / kChunks, ch = x % kChunks;
      const uint32_t pr = __shfl_sync(0xffffffffu, row, r);
      const uint32_t bytes = pr != ~0u ? 16 : 0;
      const int64_t at = (pr != ~0u ? static_cast<int64_t>(pr) * C::kRowBytes : 0) + ch * 16;
      const uint32_t to = r * C::kRowBytes + ((ch ^ (r & 7)) << 4);
      cp_async_16(kd + to, kp + at, bytes);
      cp_async_16(vd + to, vp + at, bytes);
    }
    ++issued;
    if (issued < n) {
      ld.next(p);
      rows.look_up(p, ld);
    }
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    if (s < n) issue();
    cp_async_commit();
  }

  uint32_t qf[NT][D / 16][2];
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];
  bool open = false;  // the unit's first tile of this slice has been taken
  int t_first = 0, slot = 0;
  for (int it = 0; it < n; ++it) {
    if (!open) {
      open = true;
      t_first = cur.t;
      const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hr = gr * kRowsU + nt * 8 + quad;  // head within the KV head's group
        const bool in = hr < p.g;
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(p.q) + cur.b * p.q_stride + static_cast<int64_t>(hk * p.g + hr) * D);
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
    cp_async_wait<ST - 2>();
    __syncwarp();  // tile `it` has landed for every lane, and tile it - 1 has been read by every lane
    const int s = it % ST;
    const uint32_t mask = live_mask[warp][s];
    if (issued < n) issue();
    cp_async_commit();
    const uint32_t ka = ring + s * C::kStage, va = ka + C::kTile;

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
        const int ch = 2 * kk + (lane >> 4);
        ptx::ldmatrix_x4(a0, a1, a2, a3, ka + r * C::kRowBytes + ((ch ^ (r & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16_16816(sc[ks][nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
      }
    }
    if (mask != (KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u)) {
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
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int r = ks * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        uint32_t a0, a1, a2, a3;
        const int ch = 2 * mt + ((lane >> 3) & 1);
        ptx::ldmatrix_x4_trans(a0, a1, a2, a3, va + r * C::kRowBytes + ((ch ^ (r & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16_16816(o[mt][nt], a0, a1, a2, a3, pb[ks][nt][0], pb[ks][nt][1]);
      }
    }

    const bool unit_end = cur.t == cur.tiles - 1;
    if (unit_end || it == n - 1) {
      const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
      const int heads = min(kRowsU, p.g - gr * kRowsU);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
          l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
          l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
        }
      if (unit_end && t_first == 0) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) +
                           (static_cast<int64_t>(cur.b) * p.Hq + hk * p.g + gr * kRowsU) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float i0 = l[nt][0] != 0.f ? 1.f / l[nt][0] : 0.f, i1 = l[nt][1] != 0.f ? 1.f / l[nt][1] : 0.f;
          const int hr = nt * 8 + quad;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            const uint32_t x = ptx::movmatrix_trans(ptx::pack_bf16x2(o[mt][nt][0] * i0, o[mt][nt][1] * i1));
            const uint32_t z = ptx::movmatrix_trans(ptx::pack_bf16x2(o[mt][nt][2] * i0, o[mt][nt][3] * i1));
            if (hr < heads) {
              uint32_t* yr = reinterpret_cast<uint32_t*>(y + hr * D + mt * 16);
              yr[qi] = x;
              yr[4 + qi] = z;
            }
          }
        }
      } else {
        const int64_t at = (static_cast<int64_t>(slice) * 2 + slot) * kRowsU;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int hr = nt * 8 + qi * 2 + h;
            if (hr < heads) {
              if (quad == 0) p.ml[at + hr] = make_float2(m[nt][h] * p.c, l[nt][h]);
              float* dst = p.part + (at + hr) * D;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                dst[mt * 16 + quad] = o[mt][nt][h];
                dst[mt * 16 + 8 + quad] = o[mt][nt][h + 2];
              }
            }
          }
      }
      slot = 1;  // a later unit of the slice is not its first
      open = false;
    }
    cur.next(p);
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
  const int per = scan_tiles<KT>(p, pre, warp_sum);
  const int64_t total = pre[blockDim.x] * p.units;
  const int slice = warp * gridDim.x + blockIdx.x;
  const int slices = live_slices(p, total);
  if (slice >= slices) return;
  const int64_t f0 = total * slice / slices, f1 = total * (slice + 1) / slices;
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

  Cursor<KT> ld = cursor_at<KT>(p, pre, per, f0);
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
      for (int i = lane; i < kRows * D; i += 32) {
        const int r = i / D, d = i - r * D;
        const T* q = static_cast<const T*>(p.q) + cur.b * p.q_stride + static_cast<int64_t>(hk * p.g + gr * kRows + r) * D;
        qs[i] = r < heads ? Elem<T>::load(q, d) * p.c : 0.f;
      }
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
      simt_tile<T, DPL, KT>(st, kt, kt + KT * stride, stride, qs, ps, D, lo, hi, heads);
      left = b >= 32 ? 0u : left & (~0u << b);
    }

    const bool unit_end = cur.t == cur.tiles - 1;
    if (unit_end || it == n - 1) {
      const bool whole = unit_end && t_first == 0;
      T* y = static_cast<T*>(p.y) + (static_cast<int64_t>(cur.b) * p.Hq + hk * p.g + gr * kRows) * D;
      const int64_t at = (static_cast<int64_t>(slice) * 2 + slot) * kRows;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r < heads) {
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
  const int64_t b0 = p.base[b], tiles = p.base[b + 1] - b0, total = p.base[p.B] * p.units;
  T* y = static_cast<T*>(p.y) + (static_cast<int64_t>(b) * p.Hq + h) * D;
  if (tiles == 0) {  // no key
    for (int d = tid; d < D; d += kMergeThreads) y[d] = Elem<T>::from_float(0.f);
    return;
  }
  const int slices = live_slices(p, total);
  const int64_t u0 = b0 * p.units + static_cast<int64_t>(hk * p.groups + gr) * tiles;
  // the slice that holds tile f is the last whose first tile is <= f
  const int s0 = static_cast<int>(((u0 + 1) * slices - 1) / total);
  const int s1 = static_cast<int>(((u0 + tiles) * slices - 1) / total);
  if (s0 == s1) return;  // written by the slice itself
  const int first_slot = total * s0 / slices < u0 ? 1 : 0;
  const int n = s1 - s0 + 1;
  // partial i of the unit, in rows of the workspace
  auto at = [&](int i) { return (static_cast<int64_t>(s0 + i) * 2 + (i == 0 ? first_slot : 0)) * p.rows + r; };

  float M = -INFINITY;
  for (int i = tid; i < n; i += kMergeThreads) {
    const float m = __ldcg(&p.ml[at(i)].x);
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
    L = fmaf(w, __ldcg(&p.ml[at(i)].y), L);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) L += red[1][i];

  const int cols = D / 4, subs = kMergeThreads / cols;  // D <= 512: two at least
  const int sub = tid / cols, c = tid - sub * cols;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (sub < subs) {
    auto add = [&](int i, const float4& v) {
      const float w = w_s[i];
      a.x = fmaf(w, v.x, a.x);
      a.y = fmaf(w, v.y, a.y);
      a.z = fmaf(w, v.z, a.z);
      a.w = fmaf(w, v.w, a.w);
    };
    const float4* part = reinterpret_cast<const float4*>(p.part) + c;
    int i = sub;
    for (; i + 7 * subs < n; i += 8 * subs) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = __ldcg(part + at(i + u * subs) * cols);
#pragma unroll
      for (int u = 0; u < 8; ++u) add(i + u * subs, v[u]);
    }
    for (; i < n; i += subs) add(i, __ldcg(part + at(i) * cols));
    acc_s[tid] = a;
  }
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
  size_t off_ml, off_part, bytes;
};

bool use_mma(int64_t D, int dtype) {
  return dtype == EXTKV_BF16 && (D == 64 || D == 128 || D == 256 || D == 512);
}

// Sixteen heads a unit where the KV head has more than eight and their
// accumulators fit the registers (D/4 a thread and eight heads).
int unit_rows(int64_t g, int64_t D, bool mma) { return mma && g > 8 && D <= 256 ? 16 : 8; }

int mma_warps(int64_t D) { return D <= 128 ? 8 : D == 256 ? 6 : 3; }

Plan plan_of(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  const bool mma = use_mma(D, dtype);
  Plan pl;
  const int64_t g = Hq / Hkv;
  pl.rows = unit_rows(g, D, mma);
  pl.groups = static_cast<int>((g + pl.rows - 1) / pl.rows);
  pl.warps = mma ? mma_warps(D) : kSimtWarps;
  pl.slices = std::min(num_sms() * pl.warps, kMaxSlices / pl.warps * pl.warps);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  pl.off_ml = up(sizeof(int64_t) * (B + 1));
  pl.off_part = pl.off_ml + up(sizeof(float2) * 2 * pl.slices * pl.rows);
  pl.bytes = pl.off_part + up(sizeof(float) * 2 * pl.slices * pl.rows * D);
  return pl;
}

template <class C>
cudaError_t launch_mma(const PagedParams& p, cudaStream_t s) {
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(paged_decode_mma_kernel<C>), C::kSmem);
      e != cudaSuccess)
    return e;
  PdlLaunch l(dim3(p.slices / C::WARPS), C::WARPS * 32, C::kSmem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, paged_decode_mma_kernel<C>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
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
  p.status = a.status;
  cudaError_t e;
  if (use_mma(a.D, a.dtype)) {
    *name = "paged_decode_mma";
    const bool two = pl.rows == 16;
    if (a.D == 64) e = two ? launch_mma<MmaCfg<64, 2, 32, 3, 8>>(p, a.stream) : launch_mma<MmaCfg<64, 1, 32, 3, 8>>(p, a.stream);
    else if (a.D == 128) e = two ? launch_mma<MmaCfg<128, 2, 16, 3, 8>>(p, a.stream) : launch_mma<MmaCfg<128, 1, 16, 3, 8>>(p, a.stream);
    else if (a.D == 256) e = two ? launch_mma<MmaCfg<256, 2, 16, 2, 6>>(p, a.stream) : launch_mma<MmaCfg<256, 1, 16, 2, 6>>(p, a.stream);
    else e = launch_mma<MmaCfg<512, 1, 16, 2, 3>>(p, a.stream);
  } else {
    *name = a.dtype == EXTKV_F32 ? "paged_decode_simt_f32" : "paged_decode_simt_bf16";
    e = a.dtype == EXTKV_F32 ? launch_simt_d<float>(p, a.stream) : launch_simt_d<__nv_bfloat16>(p, a.stream);
  }
  if (e != cudaSuccess) return e;
  e = a.dtype == EXTKV_F32 ? launch_merge<float>(p, a.stream) : launch_merge<__nv_bfloat16>(p, a.stream);
  if (e == cudaSuccess) note_launches(2);
  return e;
}

}  // namespace extkv
