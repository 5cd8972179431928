// shared_prefix.cu -- attention of one new token per sequence where groups of
// sequences share the pages of a prefix in front of their own.
//
// Softmax over a union of key sets is the sets' partial results (max m, sum l,
// unnormalised output O) joined: y = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// So the prefix is attended once for all rows of its group ((sequence, query head)
// of a KV head), which reads its keys once where the sequences by themselves would
// read them once each, and the sequences' own pages by the paged decode; a last
// kernel joins both.  Three launches:
//   prefix   every group's keys for all its rows; partials to the workspace
//   own      the paged decode's kernel on the axis, whole units to the workspace too; beside
//            the prefix where an SM holds both
//   join     a warp or a CTA per (sequence, query head)
// The prefixes' work is one axis of tiles as in the paged decode: (group, KV head,
// row tile) units of key tiles, cut into slices of equal cost (SliceAxis).
#include "shared_prefix.cuh"
#include "shared_prefix_tc.h"

#include <cmath>

namespace extkv {

namespace {

// ---- prefix on the SIMT lanes (fp32, other head sizes, odd pages) -----------------------

// A warp takes a slice: units of kRows rows, its keys through the ring of the paged
// decode's SIMT kernel.  Bound: the fp32 lanes, 4 D flops a row and key, and the keys again for
// every 8 rows: 16 sequences of 16 heads behind 4096, 4 KV heads of 128, fp32: 100 us (118 by the paged
// decode on tables with the prefix in front); of 8 heads of 2 KV heads of 512, bf16, behind 8192: 1049, where
// the paged decode has tensor cores and takes 53.
template <typename T, int DPL, int KT>
__global__ void __launch_bounds__(kSimtWarps * 32, 1) prefix_simt_kernel(const PrefixParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t pre[kSimtWarps * 32 + 1], warp_sum[kSimtWarps];
  __shared__ uint32_t live_mask[kSimtWarps][kSimtStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.D;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const bool few = p.G < 32;
  const GroupScan<KT> scan(p);  // (of the first groups where there are more: not used)
  int per = 0;
  int64_t mean = scan.mean;
  if (!few) per = scan_groups<KT, kSimtWarps * 32, 0>(p, pre, warp_sum, mean);
  const SliceAxis axis(p, few ? scan.total() : pre[blockDim.x], mean);
  const int slice = warp * gridDim.x + blockIdx.x;  // few tiles: one warp per SM first
  Slice<KT> sl = slice_of<KT>(p, axis, slice, [&](int64_t f) { return few ? scan.cursor(p, axis, f) : prefix_cursor<KT, kSimtWarps * 32>(p, pre, per, axis, mean, f); });
  if (!sl.more(p)) return;

  const int stride = simt_stride<T>(D);
  const int stage = 2 * KT * stride;  // elements
  uint8_t* mine = smem + warp * simt_warp_bytes<T, KT>(D);
  T* ring = reinterpret_cast<T*>(mine);
  float* qs = reinterpret_cast<float*>(mine + simt_ring_bytes<T, KT>(D));
  float* ps = qs + kRows * D;
  const int row_bytes = D * static_cast<int>(sizeof(T)), chunks = row_bytes / 16;

  Slice<KT> ahead = sl;
  PrefixCursor<KT>&cur = sl.at, &ld = ahead.at;
  uint32_t row = ~0u;  // pool row of the lane's key of tile ld
  int64_t page = -1;
  int off = 0;
  bool live = false, lead = false;
  int needed = 0, needed_of = -1;  // the first key that some row of group needed_of attends
  auto look_up = [&] {             // a tile ahead
    if (ld.g != needed_of) {
      needed_of = ld.g;
      needed = first_of_group(p, ld.group);
    }
    const int j = ld.key0() + lane;
    live = lane < KT && j >= needed && j < ld.group.hi;
    page = -1;
    if (live) {
      const int pg = j / p.page_size;
      off = j - pg * p.page_size;
      lead = lane == 0 || off == 0 || j == needed;
      page = prefix_page(p, ld.g, pg);
    }
  };
  look_up();
  int issued = 0;
  bool to_issue = true;
  auto issue = [&] {
    const int s = issued % kSimtStages;
    row = ~0u;
    if (live) {
      if (page < 0 || page >= p.num_pages) {
        if (ld.u == 0 && lead) report(p.status, EXTKV_DEV_BAD_PAGE);
      } else {
        const int64_t r = (page * p.Hkv + ld.head(p)) * p.page_size + off;
        if (EXTKV_IN_KIND(kChkPages, r, 1, p.num_pages * p.Hkv * p.page_size, p.status)) row = static_cast<uint32_t>(r);
      }
    }
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
    ld.next(p);
    to_issue = ahead.more(p);
    if (to_issue) look_up();
  };
  issue();
  cp_async_commit();

  SimtState<DPL> st;
  st.clear();
  bool open = false;
  int t_first = 0, r0 = 0, rows = 0;
  int first[kRows];  // the rows' first keys
  for (int it = 0; sl.more(p); ++it) {
    const int hk = cur.head(p);
    if (!open) {
      open = true;
      t_first = cur.t;
      st.clear();
      r0 = cur.row0(p);
      rows = min(kRows, cur.group.rows - r0);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int b = cur.group.b0 + (r0 + min(r, rows - 1)) / p.g;
        first[r] = r < rows ? first_key(p, cur.group.hi, own_length(p, b)) : 0x7fffffff;
      }
      const T* q = static_cast<const T*>(p.q);
      simt_stage_q<T, DPL>(qs, D, p.c, [&](int r) -> const T* {
        if (r >= rows) return nullptr;
        const int s = (r0 + r) / p.g, h = r0 + r - s * p.g;
        const int64_t at = (cur.group.b0 + s) * p.q_stride + static_cast<int64_t>(hk * p.g + h) * D;
        return EXTKV_IN_KIND(kChkRows, at, D, (p.B - 1) * p.q_stride + static_cast<int64_t>(p.Hq) * D, p.status) ? q + at : nullptr;
      });
    }
    __syncwarp();  // tile it - 1 has been read by every lane
    if (to_issue) issue();
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const int s = it % kSimtStages;
    const T* kt = ring + s * stage;
    const int k0 = cur.key0();
    uint32_t left = live_mask[warp][s];
    while (left) {  // runs of live keys: a bad page leaves a gap
      const int a = __ffs(left) - 1;
      const uint32_t run = ~(left >> a);
      const int b = run ? min(32, a + __ffs(run) - 1) : 32;
      int lo[kRows], hi[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        lo[r] = first[r] <= k0 ? a : first[r] - k0 >= b ? b : max(a, first[r] - k0);
        hi[r] = b;
      }
      simt_tile<T, DPL, KT>(st, kt, kt + KT * stride, stride, qs, ps, D, lo, hi);
      left = b >= 32 ? 0u : left & (~0u << b);
    }

    const bool unit_end = cur.t == cur.tiles - 1;
    if (unit_end || sl.here() == 1) {
      const bool whole = unit_end && t_first == 0;
      st.reduce();
      const int64_t at = (static_cast<int64_t>(slice) * 2 + (t_first == 0)) * kRows;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int sq = (r0 + r) / p.g, h = r0 + r - sq * p.g;
        const int64_t to = whole ? static_cast<int64_t>(cur.group.b0 + sq) * p.Hq + hk * p.g + h : at + r;
        if (r < rows && (whole ? whole_in(p, to) : slice_in(p, to, 1))) {
          if (lane == 0) (whole ? p.whole_ml : p.ml)[to] = make_float2(st.m[r], st.l[r]);
#pragma unroll
          for (int i = 0; i < DPL; ++i)
            if (lane + 32 * i < D) (whole ? p.whole : p.part)[to * D + lane + 32 * i] = st.acc[r][i];
        }
      }
      open = false;
    }
    cur.next(p);
  }
}

template <typename T, int DPL, int KT>
cudaError_t launch_simt_prefix(const PrefixParams& p, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kSimtWarps) * simt_warp_bytes<T, KT>(p.D);
  auto k = prefix_simt_kernel<T, DPL, KT>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), smem); e != cudaSuccess) return e;
  PdlLaunch l(dim3(p.slices / kSimtWarps), kSimtWarps * 32, smem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Keys of a tile of the SIMT kernels.
int simt_tile_keys(int64_t D) { return D <= 128 ? 32 : D <= 256 ? 16 : 4; }

template <typename T>
cudaError_t launch_simt_prefix_d(const PrefixParams& p, cudaStream_t s) {
  if (p.D <= 64) return launch_simt_prefix<T, 2, 32>(p, s);
  if (p.D <= 128) return launch_simt_prefix<T, 4, 32>(p, s);
  if (p.D <= 256) return launch_simt_prefix<T, 8, 16>(p, s);
  return launch_simt_prefix<T, 16, 4>(p, s);
}

// ---- the join --------------------------------------------------------------------------

struct JoinParams {
  PagedParams own;
  PrefixParams pre;
  int pre_tile;  // keys of a tile of the prefixes' axis
};

// A partial: its (max, sum) and its row.
struct Place {
  const float2* ml;
  const float* rows;
};

// Where the partials of a row's own slots lie: a whole unit's, or one of each of n slices from s on.
struct OwnParts {
  int n, s, slot, r;
  __device__ __forceinline__ OwnParts(const PagedParams& p, int64_t own0, int64_t own1, int64_t total, int hk, int hr)
      : n(0), s(0), slot(0), r(hr % p.rows) {
    if (const int64_t tiles = own1 - own0; tiles > 0) {
      const Axis axis(p, total);
      const int64_t u0 = own0 * p.units + static_cast<int64_t>(hk * p.groups + hr / p.rows) * tiles;
      s = axis.holds(u0);
      n = axis.holds(u0 + tiles - 1) - s + 1;
      slot = axis.start(s) < u0 ? 1 : 0;
    }
  }
  __device__ __forceinline__ Place at(const PagedParams& p, int64_t row, int i) const {
    if (n == 1) return own_in(p, row, 1) ? Place{p.own_ml + row, p.own_part + row * p.D} : Place{nullptr, nullptr};
    const int64_t x = (static_cast<int64_t>(s + i) * 2 + (i == 0 ? slot : 0)) * p.rows + r;
    return part_in(p, x, 1, static_cast<int64_t>(p.slices) * 2) ? Place{p.ml + x, p.part + x * p.D} : Place{nullptr, nullptr};
  }
};

// Four elements of a row as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// A row and its result by one warp, from keys [lo, hi) of group g's prefix and its own slots' partials.  The
// prefix' kernels multiply a row of V by the weights of all rows of a unit, by 0 for those that do not attend
// it, which an infinity or a NaN turns into NaN: rows that this can have reached are attended again here,
// with their own keys alone.  Slow, since a warp takes key after key, and only for such rows: 64 sequences of 32
// heads, windows of 4096 behind 8192, an infinity that some of them attend: 1.3 ms, 61 us with finite pages.
template <typename T, int VPL>
__device__ __noinline__ void attend_alone(const JoinParams& jp, int g, int b, int h, int lo, int hi, OwnParts own) {
  const PagedParams& p = jp.own;
  const PrefixParams& f = jp.pre;
  constexpr int kAhead = VPL == 1 ? 4 : 2;
  const int lane = threadIdx.x & 31, D = f.D, hk = h / f.g;
  const int64_t y_row = static_cast<int64_t>(b) * f.Hq + h;
  const int64_t q_at = b * f.q_stride + static_cast<int64_t>(h) * D;
  const bool q_in = EXTKV_IN_KIND(kChkRows, q_at, D, (f.B - 1) * f.q_stride + static_cast<int64_t>(f.Hq) * D, f.status);
  float M = -INFINITY, L = 0.f;
  float4 q[VPL], a[VPL];
  int at[VPL];  // the lane's columns; -1: none
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    at[v] = lane + 32 * v < D / 4 ? 4 * (lane + 32 * v) : -1;
    q[v] = at[v] >= 0 && q_in ? load4(static_cast<const T*>(f.q) + q_at + at[v]) : make_float4(0.f, 0.f, 0.f, 0.f);
    q[v] = make_float4(q[v].x * f.c, q[v].y * f.c, q[v].z * f.c, q[v].w * f.c);
    a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // (max m, sum l, columns x) joined to the row's
  auto add = [&](float m, float l, const float4 (&x)[VPL]) {
    const float mn = fmaxf(M, m), ref = mn == -INFINITY ? 0.f : mn;
    const float old = M == -INFINITY ? 0.f : ptx::ex2(M - ref), w = m == -INFINITY ? 0.f : ptx::ex2(m - ref);
    M = mn;
    L = fmaf(w, l, L * old);
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      a[v] = make_float4(fmaf(w, x[v].x, a[v].x * old), fmaf(w, x[v].y, a[v].y * old), fmaf(w, x[v].z, a[v].z * old),
                         fmaf(w, x[v].w, a[v].w * old));
  };
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int n = min(32, hi - j0);
    int64_t row = -1;
    if (lane < n) {
      const int pg = (j0 + lane) / f.page_size, off = j0 + lane - pg * f.page_size;
      const int64_t page = prefix_page(f, g, pg);
      if (page >= 0 && page < f.num_pages) row = (page * f.Hkv + hk) * f.page_size + off;
      if (row >= 0 && !EXTKV_IN_KIND(kChkPages, row, 1, f.num_pages * f.Hkv * f.page_size, f.status)) row = -1;
    }
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      int64_t pr[kAhead];
      float4 k[kAhead][VPL], x[kAhead][VPL];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        pr[i] = __shfl_sync(0xffffffffu, row, i0 + i);  // 32 % kAhead == 0; -1 behind the last key
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const bool in = pr[i] >= 0 && at[v] >= 0;
          k[i][v] = in ? load4(static_cast<const T*>(f.k) + pr[i] * D + at[v]) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[i][v] = in ? load4(static_cast<const T*>(f.v) + pr[i] * D + at[v]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (pr[i] < 0) continue;  // (the warp's)
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          s = fmaf(q[v].x, k[i][v].x, fmaf(q[v].y, k[i][v].y, fmaf(q[v].z, k[i][v].z, fmaf(q[v].w, k[i][v].w, s))));
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        add(s, 1.f, x[i]);
      }
    }
  }
  for (int i = 0; i < own.n; ++i) {
    const Place mine = own.at(p, y_row, i);
    if (!mine.ml) continue;
    const float2 ml = __ldcg(mine.ml);
    float4 x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      x[v] = at[v] >= 0 ? __ldcg(reinterpret_cast<const float4*>(mine.rows + at[v])) : make_float4(0.f, 0.f, 0.f, 0.f);
    add(ml.x, ml.y, x);
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  if (!y_in(p, y_row * D, D)) return;
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (at[v] >= 0) store4(static_cast<T*>(p.y) + y_row * D + at[v], a[v], inv);
}

// WPR warps take one (sequence, query head).  Its partials, in order: those of its
// prefix (a whole unit's, or one of each slice that holds tiles of the unit), then those
// of its own pages likewise.  A warp takes a run of them, 32 at a time: a lane each
// for the weights, then 4 * VPL columns a lane; several warps are joined in order.  Bound:
// latency, three rounds of dependent loads; a warp a row where there are rows for the GPU
// (64 sequences of 32 heads behind 8191 keys: 7 us, 26 with a CTA a row).
constexpr int kJoinWarps = 8;

// WINDOW: the call has one.
template <typename T, int VPL, int WPR, bool WINDOW>
__global__ void __launch_bounds__(kJoinWarps * 32) prefix_join_kernel(const __grid_constant__ JoinParams jp) {
  __shared__ float2 ml_s[kJoinWarps];
  __shared__ float4 acc_s[WPR > 1 ? kJoinWarps : 1][WPR > 1 ? VPL * 32 : 1];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const PagedParams& p = jp.own;
  const PrefixParams& f = jp.pre;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.D;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinWarps / WPR) + warp / WPR;
  if (row >= static_cast<int64_t>(p.B) * p.Hq) return;  // (whole warps; WPR > 1: none)
  const int b = static_cast<int>(row / p.Hq), h = static_cast<int>(row - static_cast<int64_t>(b) * p.Hq);
  const int hk = h / p.g, hr = h - hk * p.g;
  auto pre_base = [&](int g) {
    return EXTKV_IN_KIND(kChkPartial, g, 1, static_cast<int64_t>(f.G) + 2, f.status) ? f.base[g] : 0;
  };
  const int ok = *f.ok;
  const int64_t n_own = length_of(p, b), pre_total = pre_base(f.G), mean = pre_base(f.G + 1);
  int64_t own0 = 0, own1 = 0, own_total = 0;
  if (base_in(p, b) && base_in(p, b + 1)) {
    own0 = p.base[b];
    own1 = p.base[b + 1];
    own_total = p.base[p.B] * p.units;
  }
  // the group: the last with cu[g] <= b < cu[g + 1], 32 candidates at a time
  int g = -1;
  for (int lo = 0, hi = f.G + 1; lo < hi;) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && cu_of(f, at) <= b));
    if (n == 0) break;
    g = lo + (n - 1) * step;
    hi = min(hi, g + step);
    lo = g + 1;
    if (step == 1) break;
  }
  if (!ok) return;  // the groups are not in order: nothing is written
  bool bad = n_own < 0 || n_own > static_cast<int64_t>(p.max_pages) * p.page_size;
  // the prefix' partials
  int n_pre = 0, s_pre = 0, r_pre = 0;
  int first = 0, end = 0;  // the keys of the prefix that the row attends
  if (g >= 0 && g < f.G) {
    const int64_t b0 = pre_base(g);
    const Group gr = group_at(f, g);
    bad |= gr.bad;
    const int tiles = gr.lo < gr.hi ? (gr.hi + jp.pre_tile - 1) / jp.pre_tile - gr.lo / jp.pre_tile : 0;
    if (tiles) {
      const int r = (b - gr.b0) * p.g + hr;
      const SliceAxis axis(f, pre_total, mean);
      const int cost = cost_of(tiles, mean);
      const int2 parts = axis.parts(b0 + (static_cast<int64_t>(hk) * gr.row_tiles(f) + r / f.rows) * (tiles + cost), tiles, cost);
      s_pre = parts.x;
      n_pre = parts.y;
      r_pre = r % f.rows;
      first = first_key(f, gr.hi, n_own);
      end = gr.hi;
    }
  }
  const OwnParts own(p, own0, own1, own_total, hk, hr);
  const int n = bad ? 0 : n_pre + own.n;
  auto at = [&](int i) -> Place {
    if (i >= n_pre) return own.at(p, row, i - n_pre);
    if (n_pre == 1) return whole_in(f, row) ? Place{f.whole_ml + row, f.whole + row * D} : Place{nullptr, nullptr};
    const int64_t x = (static_cast<int64_t>(s_pre + i) * 2 + (i == 0)) * f.rows + r_pre;
    return slice_in(f, x, 1) ? Place{f.ml + x, f.part + x * D} : Place{nullptr, nullptr};
  };

  const int part = warp % WPR, i0 = n * part / WPR, i1 = n * (part + 1) / WPR;
  float M = -INFINITY, L = 0.f;
  float4 a[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = i0; c0 < i1; c0 += 32) {
    const int m = min(32, i1 - c0);
    const Place mine = lane < m ? at(c0 + lane) : Place{nullptr, nullptr};
    const float2 ml = mine.ml ? __ldcg(mine.ml) : make_float2(-INFINITY, 0.f);
    const int64_t rows = reinterpret_cast<int64_t>(mine.rows);
    constexpr int kAhead = VPL == 1 ? 8 : 8 / VPL;
    float4 x[kAhead][VPL];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float4* src = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, rows, min(j0 + u, 31)));
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          x[u][v] = j0 + u < m && src && lane + 32 * v < D / 4 ? __ldcg(src + lane + 32 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    fetch(0);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float mn = fmaxf(M, top), ref = mn == -INFINITY ? 0.f : mn;
    const float old = M == -INFINITY ? 0.f : ptx::ex2(M - ref);
    const float w = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - ref);  // -inf: no key of the partial is attended
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    L = fmaf(L, old, l);
    M = mn;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      a[v].x *= old;
      a[v].y *= old;
      a[v].z *= old;
      a[v].w *= old;
    }
    for (int j0 = 0; j0 < m; j0 += kAhead) {
      if (j0) fetch(j0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, min(j0 + u, 31));
        if (j0 + u < m) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            a[v].x = fmaf(wu, x[u][v].x, a[v].x);
            a[v].y = fmaf(wu, x[u][v].y, a[v].y);
            a[v].z = fmaf(wu, x[u][v].z, a[v].z);
            a[v].w = fmaf(wu, x[u][v].w, a[v].w);
          }
        }
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) ml_s[warp] = make_float2(M, L);
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc_s[warp][lane + 32 * v] = a[v];
    __syncthreads();
    if (warp) return;
    M = -INFINITY;
#pragma unroll
    for (int k = 0; k < WPR; ++k) M = fmaxf(M, ml_s[k].x);
    const float ref = M == -INFINITY ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < WPR; ++k) {
      const float w = ml_s[k].x == -INFINITY ? 0.f : ptx::ex2(ml_s[k].x - ref);
      L = fmaf(w, ml_s[k].y, L);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const float4 z = acc_s[k][lane + 32 * v];
        a[v].x = fmaf(w, z.x, a[v].x);
        a[v].y = fmaf(w, z.y, a[v].y);
        a[v].z = fmaf(w, z.z, a[v].z);
        a[v].w = fmaf(w, z.w, a[v].w);
      }
    }
  }
  if (WINDOW && first > 0 && n > 0) {  // its window leaves keys out that others of its group may attend
    bool odd = false;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      odd |= !(fabsf(a[v].x) < INFINITY && fabsf(a[v].y) < INFINITY && fabsf(a[v].z) < INFINITY && fabsf(a[v].w) < INFINITY);
    if (__any_sync(0xffffffffu, odd)) {
      if constexpr (WINDOW) attend_alone<T, VPL>(jp, g, b, h, first, end, own);
      return;
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;  // no key: a zero row
  const int64_t y_at = row * D;
  if (!y_in(p, y_at, D)) return;
  T* y = static_cast<T*>(p.y) + y_at;
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (lane + 32 * v < D / 4) store4(y + 4 * (lane + 32 * v), a[v], inv);
}

template <typename T, int VPL>
cudaError_t launch_join_d(const JoinParams& jp, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(jp.own.B) * jp.own.Hq;
  // a warp a row where that fills a good part of the GPU's warps, else a CTA a row
  const bool many = rows >= int64_t(num_sms()) * 4;
  PdlLaunch l(dim3(static_cast<unsigned>(many ? (rows + kJoinWarps - 1) / kJoinWarps : rows)), kJoinWarps * 32, 0, s);
  auto go = [&](auto one, auto several) { return cudaLaunchKernelEx(&l.cfg, many ? one : several, jp); };
  cudaError_t e = jp.pre.window > 0 ? go(prefix_join_kernel<T, VPL, 1, true>, prefix_join_kernel<T, VPL, kJoinWarps, true>)
                                    : go(prefix_join_kernel<T, VPL, 1, false>, prefix_join_kernel<T, VPL, kJoinWarps, false>);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_join(const JoinParams& jp, cudaStream_t s) {
  return jp.own.D <= 128 ? launch_join_d<T, 1>(jp, s) : jp.own.D <= 256 ? launch_join_d<T, 2>(jp, s) : launch_join_d<T, 4>(jp, s);
}

// ---- host ------------------------------------------------------------------------------

struct PrefixPlan {
  Plan own;
  int rows, slices;
  size_t off_own_ml, off_own, off_ok, off_base, off_ml, off_part, off_whole_ml, off_whole, bytes;
};

// Own pages in CTAs small enough, in registers (a warp on each of an SM's four parts) and rings,
// to share an SM with one of the prefix; three an SM once it is done.  (Head size 128 and units of 8
// heads; not built for others.)
constexpr int kBesideWarps = 4, kBesideCtas = 3;
bool can_run_beside(int64_t g, int64_t D, bool tc) { return tc && D == 128 && unit_rows(g, D, true) == 8; }

// Whether they do.  Beside it the two overlap, after it each is faster: a prefix of many
// rows loses issue slots to a kernel that waits for memory.  So where rows are few, or
// the own keys are most of the work, by what the tables can hold (lengths are on the
// device): a tile of a unit takes about 1 us of an SM, own keys what their bytes take.
// 64 sequences of at most 1024 own keys behind 8191 (256 rows): 53 us beside, 74 after; 2
// sequences behind 30000 (8 rows) 53 and 58; 68 of at most 304 behind 8000 (238 rows) 53 and
// 47; 225 of 128 behind 32768 (450 rows) 157 and 132.
bool own_beside(const SharedPrefixArgs& a, bool tc) {
  const PagedDecodeArgs& d = a.own;
  if (!can_run_beside(d.Hq / d.Hkv, d.D, tc) || a.G == 0) return false;
  const double rows = static_cast<double>(d.B) * (d.Hq / d.Hkv) / a.G;  // of a group and KV head
  const double tiles = static_cast<double>(a.G) * d.Hkv * std::ceil(rows / prefix_tc_rows(d.D)) * a.max_prefix_pages * d.page_size / prefix_tc_tile_keys();
  const double prefix_us = tiles / num_sms();
  const double own_us = static_cast<double>(d.B) * d.Hkv * d.max_pages * d.page_size * d.D * 4 / 6.8e6;
  return rows <= 64 || prefix_us <= own_us / 2;
}

// tc: the prefix on the tensor cores.  beside: own pages beside it.
PrefixPlan prefix_plan(int64_t B, int64_t G, int64_t Hq, int64_t Hkv, int64_t D, int dtype, bool tc, bool beside) {
  PrefixPlan pl;
  pl.own = beside ? plan_with(B, Hq / Hkv, D, true, 8, kBesideWarps, kBesideCtas) : plan_of(B, Hq, Hkv, D, dtype);
  pl.rows = tc ? prefix_tc_rows(D) : kRows;
  pl.slices = tc ? std::min(num_sms(), kMaxSlices) : std::min(num_sms() * kSimtWarps, kMaxSlices / kSimtWarps * kSimtWarps);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t rows = static_cast<size_t>(B) * Hq, parts = static_cast<size_t>(pl.slices) * 2 * pl.rows;
  size_t at = up(pl.own.bytes);
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += up(bytes);
    return x;
  };
  pl.off_own_ml = take(sizeof(float2) * rows);
  pl.off_own = take(sizeof(float) * rows * D);
  pl.off_ok = take(sizeof(int));
  pl.off_base = take(sizeof(int64_t) * (G + 2));
  pl.off_ml = take(sizeof(float2) * parts);
  pl.off_part = take(sizeof(float) * parts * D);
  pl.off_whole_ml = take(sizeof(float2) * rows);
  pl.off_whole = take(sizeof(float) * rows * D);
  pl.bytes = at;
  return pl;
}

template <int D, int NT, int KT, int SLOTS, int WARPS>
cudaError_t launch_own(PagedParams& p, cudaStream_t s) {
  return tma_pages(p, D, 2) ? launch_mma_cfg<MmaCfg<D, NT, KT, SLOTS, WARPS, true, false, true>>(p, s)
                            : launch_mma_cfg<MmaCfg<D, NT, KT, SLOTS, WARPS, false, false, true>>(p, s);
}

cudaError_t launch_own_beside(PagedParams& p, cudaStream_t s) {
  return launch_mma_cfg<MmaCfg<128, 1, 16, 4, kBesideWarps, false, false, true, 2, 1, kBesideCtas>>(p, s);
}

}  // namespace

size_t shared_prefix_workspace_bytes(int64_t B, int64_t G, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  // (whatever the pages and the tables' widths are)
  size_t most = prefix_plan(B, G, Hq, Hkv, D, dtype, false, false).bytes;
  if (prefix_tc_supported(D, dtype, 16)) most = std::max(most, prefix_plan(B, G, Hq, Hkv, D, dtype, true, false).bytes);
  if (can_run_beside(Hq / Hkv, D, prefix_tc_supported(D, dtype, 16)))
    most = std::max(most, prefix_plan(B, G, Hq, Hkv, D, dtype, true, true).bytes);
  return most;
}

cudaError_t launch_shared_prefix(const SharedPrefixArgs& a, const char** name) {
  const PagedDecodeArgs& d = a.own;
  const bool tc = prefix_tc_supported(d.D, d.dtype, d.page_size);
  const bool beside = own_beside(a, tc);
  const PrefixPlan pl = prefix_plan(d.B, a.G, d.Hq, d.Hkv, d.D, d.dtype, tc, beside);
  uint8_t* ws = static_cast<uint8_t*>(d.workspace);
  JoinParams jp{};
  PagedParams& p = jp.own;
  p = params_of(d, pl.own);
  p.own_ml = reinterpret_cast<float2*>(ws + pl.off_own_ml);
  p.own_part = reinterpret_cast<float*>(ws + pl.off_own);
  PrefixParams& f = jp.pre;
  f.q = d.q;
  f.k = d.k_pages;
  f.v = d.v_pages;
  f.table = a.prefix_table;
  f.len = a.prefix_len;
  f.cu = a.cu_groups;
  f.nonpad = d.nonpad;
  f.c = p.c;
  f.window = p.window;
  f.B = p.B;
  f.G = static_cast<int>(a.G);
  f.Hq = p.Hq;
  f.Hkv = p.Hkv;
  f.g = p.g;
  f.D = p.D;
  f.page_size = p.page_size;
  f.max_pages = static_cast<int>(a.max_prefix_pages);
  f.num_pages = p.num_pages;
  f.q_stride = p.q_stride;
  f.own_cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  f.rows = pl.rows;
  f.slices = pl.slices;
  f.full = tc && static_cast<int64_t>(p.B) * p.g >= 128 * a.G;
  f.wait_limit = p.wait_limit;
  f.ok = reinterpret_cast<int*>(ws + pl.off_ok);
  f.base = reinterpret_cast<int64_t*>(ws + pl.off_base);
  f.ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  f.part = reinterpret_cast<float*>(ws + pl.off_part);
  f.whole_ml = reinterpret_cast<float2*>(ws + pl.off_whole_ml);
  f.whole = reinterpret_cast<float*>(ws + pl.off_whole);
  f.status = d.status;
  const bool f32 = d.dtype == EXTKV_F32;
  *name = tc ? "shared_prefix_tcgen05" : f32 ? "shared_prefix_simt_f32" : "shared_prefix_simt_bf16";
  if (!beside && can_run_beside(p.g, d.D, tc)) *name = "shared_prefix_tcgen05_after";
  cudaError_t e = tc    ? launch_prefix_tc(f, d.stream)
                  : f32 ? launch_simt_prefix_d<float>(f, d.stream)
                        : launch_simt_prefix_d<__nv_bfloat16>(f, d.stream);
  if (e != cudaSuccess) return e;
  jp.pre_tile = tc ? prefix_tc_tile_keys() : simt_tile_keys(d.D);
  if (use_mma(d.D, d.dtype)) {
    const bool two = pl.own.rows == 16;
    if (beside) e = launch_own_beside(p, d.stream);
    else if (d.D == 64) e = two ? launch_own<64, 2, 32, 8, 6>(p, d.stream) : launch_own<64, 1, 32, 8, 6>(p, d.stream);
    else if (d.D == 128) e = two ? launch_own<128, 2, 32, 4, 6>(p, d.stream) : launch_own<128, 1, 32, 4, 6>(p, d.stream);
    else if (d.D == 256) e = two ? launch_own<256, 2, 16, 6, 4>(p, d.stream) : launch_own<256, 1, 16, 6, 4>(p, d.stream);
    else e = launch_own<512, 1, 16, 2, 6>(p, d.stream);
  } else {
    e = f32 ? launch_simt_d<float, float, true>(p, d.stream) : launch_simt_d<__nv_bfloat16, __nv_bfloat16, true>(p, d.stream);
  }
  if (e != cudaSuccess) return e;
  e = f32 ? launch_join<float>(jp, d.stream) : launch_join<__nv_bfloat16>(jp, d.stream);
  if (e == cudaSuccess) note_launches(3);
  return e;
}

}  // namespace extkv
