// shared_prefix.cuh -- groups of sequences that share a prefix: the prefixes' work
// as one axis of tiles, and where a row's partial results lie.
#pragma once

#include "paged_decode.cuh"

namespace extkv {

struct PrefixParams {
  const void* q;
  const void* k;
  const void* v;
  const int64_t* table;   // [G][max_pages] the prefixes' pages
  const int64_t* len;     // [G]
  const int64_t* cu;      // [G + 1] the groups' sequences
  const int64_t* nonpad;  // [B] the sequences' own slots
  float c;                // scale * log2(e)
  int window, B, G, Hq, Hkv, g, D, page_size, max_pages;
  int64_t num_pages, q_stride, own_cap;  // own_cap: slots of a sequence's own table
  int rows;     // rows ((sequence, query head) of a KV head) per unit
  int slices;   // pieces the axis is cut into: CTAs (tensor cores) or warps
  int full;     // groups fill a good part of a unit's rows
  int box;      // rows of a TMA request
  int q_tma;    // q's rows come by TMA
  uint32_t wait_limit;
  int* ok;      // written by the prefix kernel: 1 where cu is in order
  int64_t* base;    // [G + 1] cells before each group, then the mean slice (SliceAxis)
  float2* ml;       // [slices][2][rows] (max in log2 units, sum) of a slice's parts of units begun before it, and in it
  float* part;      // [slices][2][rows][D]
  float2* whole_ml; // [B * Hq] units that lie in one slice
  float* whole;     // [B * Hq][D]
  int32_t* status;
};

// One group: its rows per KV head, and the keys [lo, hi) that some row may attend
// (a row of window W attends no key below hi + own length - W).
struct Group {
  int b0, rows, lo, hi;
  bool bad;  // a length outside the table
  __device__ __forceinline__ int row_tiles(const PrefixParams& p) const { return (rows + p.rows - 1) / p.rows; }
  template <int KT>
  __device__ __forceinline__ int tiles() const {
    return lo < hi ? (hi + KT - 1) / KT - lo / KT : 0;
  }
};

__device__ __forceinline__ int64_t cu_of(const PrefixParams& p, int g) {
  return EXTKV_IN_KIND(kChkLens, g, 1, static_cast<int64_t>(p.G) + 1, p.status) ? p.cu[g] : 0;
}

// (of a cu that is in order)
__device__ __forceinline__ Group group_at(const PrefixParams& p, int g) {
  Group r;
  r.b0 = static_cast<int>(cu_of(p, g));
  r.rows = (static_cast<int>(cu_of(p, g + 1)) - r.b0) * p.g;
  const int64_t n = EXTKV_IN_KIND(kChkLens, g, 1, p.G, p.status) ? p.len[g] : 0;
  r.bad = n < 0 || n > static_cast<int64_t>(p.max_pages) * p.page_size;
  r.hi = r.bad ? 0 : static_cast<int>(n);
  r.lo = p.window > 0 && r.hi > p.window ? r.hi - p.window : 0;
  return r;
}

// The first prefix key that a sequence with n own slots behind a prefix of P attends
// (P: none, as for a length outside its table, whose row is zero).
__device__ __forceinline__ int first_key(const PrefixParams& p, int P, int64_t n) {
  if (n < 0 || n > p.own_cap) return P;
  if (p.window <= 0) return 0;
  const int64_t lo = static_cast<int64_t>(P) + n - p.window;
  return lo <= 0 ? 0 : lo >= P ? P : static_cast<int>(lo);
}

__device__ __forceinline__ int64_t own_length(const PrefixParams& p, int b) {
  return EXTKV_IN_KIND(kChkLens, b, 1, p.B, p.status) ? p.nonpad[b] : 0;
}

// The first prefix key that some row of the group attends; the warp's lanes together.
__device__ __forceinline__ int first_of_group(const PrefixParams& p, const Group& g) {
  if (p.window <= 0) return 0;
  int x = g.hi;
  for (int b = threadIdx.x & 31; b < g.rows / p.g; b += 32) x = min(x, first_key(p, g.hi, own_length(p, g.b0 + b)));
  return __reduce_min_sync(0xffffffffu, x);
}

__device__ __forceinline__ int64_t prefix_page(const PrefixParams& p, int g, int pg) {
  const int64_t at = static_cast<int64_t>(g) * p.max_pages + pg;
  return EXTKV_IN_KIND(kChkTable, at, 1, static_cast<int64_t>(p.G) * p.max_pages, p.status) ? p.table[at] : -1;
}

__device__ __forceinline__ bool slice_in(const PrefixParams& p, int64_t at, int rows) {
  return EXTKV_IN_KIND(kChkPartial, at, rows, static_cast<int64_t>(p.slices) * 2 * p.rows, p.status);
}
__device__ __forceinline__ bool whole_in(const PrefixParams& p, int64_t row) {
  return EXTKV_IN_KIND(kChkPartial, row, 1, static_cast<int64_t>(p.B) * p.Hq, p.status);
}

// The axis cut into slices.  It counts cells: a unit's tiles, and before a unit of
// fewer tiles than a slice kCost more, since a slice that holds several units pays for
// each (its q, its partial rows: about as long as kCost tiles of the tensor-core
// kernel).  Slices end at multiples of total / n; an end that is `snap` tiles or fewer from the
// start or end of its unit is moved there, which saves a part.
//
// There are as many slices as SMs (or warps) where rows are few.  Where they fill units each
// slice leaves as many partial rows, which it writes and the join reads: n slices then cost total / n
// tiles and, in the end, about n / 4, least at n = 2 sqrt(total).  Own pages beside the prefix get
// the SMs left over.  64 sequences of 4 heads a KV head behind 8191 keys (1024 tiles): 60 us with 152
// slices, 55 with 85, 53 with 64, 66 with 43.  So many at most, and as many as SMs (us a call behind a
// flush of L2): 64 sequences of 32 heads, 8 KV heads, behind 8191, own slots up to 100 / 1000, head size 128 48
// and 63 / 73 and 74, 64 43 and 54 / 71 and 70, 256 (16 heads, 4 KV heads) 46 and 62 / 86 and 89; 32 of 32 heads, 2
// KV heads of 128, behind 16384 48 and 58 / 49 and 63; 64 of 4 heads, one KV head, behind 131072 58 and
// 68 (head size 64, behind 65536, 43 and 52); 32 of them, head size 256, behind 65536 48 and 60; 32 of 32 heads,
// 8 KV heads, behind 8191 (128 rows) 42 and 48; four groups of 64 behind 2000 75 and 75.
constexpr int kCost = 6;
struct SliceAxis {
  int64_t total;
  int n, snap;
  // mean: tiles of the axis over the slices there are
  __device__ __forceinline__ SliceAxis(const PrefixParams& p, int64_t total_, int64_t mean)
      : total(total_), n(slices_of(p, total_)), snap(static_cast<int>(mean / 2 < kCost ? mean / 2 : kCost)) {}
  static __device__ __forceinline__ int slices_of(const PrefixParams& p, int64_t total) {
    const int most = p.full ? min(p.slices, max(1, static_cast<int>(2.f * sqrtf(static_cast<float>(total))))) : p.slices;
    return total < most ? static_cast<int>(total) : most;
  }
  __device__ __forceinline__ int64_t end(int i) const { return i >= n ? total : Axis::div(i * total, n); }
  // the first slice that ends (as cut) at cell f or behind it; f >= 0
  __device__ __forceinline__ int behind(int64_t f) const {
    const int64_t x = Axis::div(f * n + total - 1, total);
    return x < n ? static_cast<int>(x) : n;
  }
  // A unit of `tiles` tiles that begins at cell u0 (its cost first): the slice of its first part, and how many parts.
  __device__ __forceinline__ int2 parts(int64_t u0, int tiles, int cost) const {
    const int64_t lo = u0 + cost + (snap + 1 < tiles ? snap + 1 : tiles), hi = u0 + cost + tiles - snap;  // ends in [lo, hi) cut the unit
    const int a = behind(lo);
    return make_int2(a - 1, 1 + (lo < hi ? behind(hi) - a : 0));
  }
};
__device__ __forceinline__ int cost_of(int tiles, int64_t mean) { return tiles < mean ? kCost : 0; }

// A position on the axis: tile t of unit u (KV head, then row tile) of group g.
template <int KT>
struct PrefixCursor {
  int g, u, t, tiles, row_tiles;
  Group group;
  __device__ __forceinline__ int key0() const { return (group.lo / KT + t) * KT; }
  __device__ __forceinline__ int head(const PrefixParams&) const { return u / row_tiles; }
  __device__ __forceinline__ int row0(const PrefixParams& p) const { return (u % row_tiles) * p.rows; }
  __device__ __forceinline__ void load(const PrefixParams& p) {
    group = group_at(p, g);
    tiles = group.tiles<KT>();
    row_tiles = group.row_tiles(p);
  }
  // at cell `rest` of the group
  __device__ __forceinline__ void place(const SliceAxis&, int64_t mean, int64_t rest) {
    const int cost = cost_of(tiles, mean);
    u = static_cast<int>(Axis::div(rest, tiles + cost));
    t = max(0, static_cast<int>(rest - static_cast<int64_t>(u) * (tiles + cost)) - cost);
  }
  // a slice's end: to the unit's start or the next unit's where that is near
  __device__ __forceinline__ void snap(const PrefixParams& p, const SliceAxis& axis) {
    if (t <= axis.snap) t = 0;
    else if (tiles - t <= axis.snap) next_unit(p);
  }
  // the next unit, at its first tile
  __device__ __forceinline__ void next_unit(const PrefixParams& p) {
    t = 0;
    if (++u < row_tiles * p.Hkv) return;
    u = 0;
    do {
      if (++g >= p.G) return;
      load(p);
    } while (tiles == 0 || row_tiles == 0);
  }
  __device__ __forceinline__ void next(const PrefixParams& p) {
    if (++t == tiles) next_unit(p);
  }
};

// Cells of a group (mean < 0: tiles alone).
template <int KT>
__device__ __forceinline__ int64_t cells_of_group(const PrefixParams& p, const Group& g, int64_t mean) {
  const int tiles = g.tiles<KT>();
  return tiles ? static_cast<int64_t>(tiles + cost_of(tiles, mean)) * g.row_tiles(p) * p.Hkv : 0;
}

// Block-wide: the cells before each chunk of groups, and their total (0 where cu is
// not in order, which block 0 flags), and the mean slice.  Block 0 also leaves every
// group's base, the mean and `ok` for the join.  The block's first NT threads take part,
// and meet at barrier ID; `pre` has NT + 1 entries.
template <int ID, int NT>
__device__ __forceinline__ void meet() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(NT) : "memory");
}
template <int ID, int NT>
__device__ __forceinline__ bool meet_or(bool x) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\tbar.red.or.pred b, %2, %3, a;\n\tselp.b32 %0, 1, 0, b;\n\t}"
               : "=r"(any)
               : "r"(static_cast<uint32_t>(x)), "n"(ID), "n"(NT)
               : "memory");
  return any;
}
template <int KT, int NT, int ID>
__device__ __forceinline__ int scan_groups(const PrefixParams& p, int64_t* pre, int64_t* warp_sum, int64_t& mean) {
  constexpr int nt = NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.G + nt - 1) / nt;
  const int g0 = min(p.G, tid * per), g1 = min(p.G, g0 + per);
  bool bad = false;
  for (int g = g0; g < g1; ++g) {
    const int64_t a = cu_of(p, g), b = cu_of(p, g + 1);
    bad |= a < 0 || b < a || b > p.B;
  }
  bad = meet_or<ID, NT>(bad);
  mean = -1;
  for (int pass = 0; pass < 2; ++pass) {  // tiles, then cells
    int64_t sum = 0;
    if (!bad)
      for (int g = g0; g < g1; ++g) sum += cells_of_group<KT>(p, group_at(p, g), mean);
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    meet<ID, NT>();
    int64_t off = 0;
    for (int w = 0; w < warp; ++w) off += warp_sum[w];
    pre[tid] = off + inc - sum;
    if (tid == nt - 1) pre[nt] = off + inc;
    meet<ID, NT>();
    if (pass == 0) {
      mean = Axis::div(pre[nt], p.slices);
      meet<ID, NT>();
    }
  }
  if (blockIdx.x == 0) {
    if (tid == 0) {
      *p.ok = bad ? 0 : 1;
      if (bad) report(p.status, EXTKV_DEV_BAD_SEQLENS);
    }
    auto base = [&](int g, int64_t at) {
      if (EXTKV_IN_KIND(kChkPartial, g, 1, static_cast<int64_t>(p.G) + 2, p.status)) p.base[g] = at;
    };
    int64_t at = pre[tid];
    if (!bad)
      for (int g = g0; g < g1; ++g) {
        base(g, at);
        const Group gr = group_at(p, g);
        at += cells_of_group<KT>(p, gr, mean);
        if (gr.bad) report(p.status, EXTKV_DEV_BAD_NONPAD);
      }
    if (tid == nt - 1 && !bad) {
      base(p.G, pre[nt]);
      base(p.G + 1, mean);
    }
  }
  return per;
}

// The same for at most 31 groups, a lane each: every warp scans them for itself, without
// meeting the block.
template <int KT>
struct GroupScan {
  Group group;  // lane g's
  int tiles, row_tiles;
  int64_t end, mean;  // cells up to and with this lane's group; the mean slice
  bool bad;           // cu is not in order
  __device__ __forceinline__ explicit GroupScan(const PrefixParams& p) {
    const int lane = threadIdx.x & 31;
    const int64_t at = lane <= p.G ? cu_of(p, lane) : 0, len = lane < p.G && EXTKV_IN_KIND(kChkLens, lane, 1, p.G, p.status) ? p.len[lane] : 0;
    const int64_t to = __shfl_down_sync(0xffffffffu, at, 1);
    const bool mine = lane < p.G;
    bad = __any_sync(0xffffffffu, mine && (at < 0 || to < at || to > p.B));
    group.b0 = static_cast<int>(at);
    group.rows = mine && !bad ? (static_cast<int>(to) - group.b0) * p.g : 0;
    group.bad = len < 0 || len > static_cast<int64_t>(p.max_pages) * p.page_size;
    group.hi = group.bad ? 0 : static_cast<int>(len);
    group.lo = p.window > 0 && group.hi > p.window ? group.hi - p.window : 0;
    tiles = group.tiles<KT>();
    row_tiles = group.row_tiles(p);
    const int64_t units = static_cast<int64_t>(row_tiles) * p.Hkv;
    mean = tiles * units;
#pragma unroll
    for (int o = 16; o; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
    mean = Axis::div(mean, p.slices);
    const int64_t n = tiles ? (tiles + cost_of(tiles, mean)) * units : 0;
    end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    if (p.G < 32 && blockIdx.x == 0 && threadIdx.x < 32) {
      if (lane == 0) {
        *p.ok = bad ? 0 : 1;
        if (bad) report(p.status, EXTKV_DEV_BAD_SEQLENS);
      }
      if (lane <= p.G && EXTKV_IN_KIND(kChkPartial, lane, 2, static_cast<int64_t>(p.G) + 2, p.status)) {
        p.base[lane] = end - n;
        if (lane == p.G) p.base[lane + 1] = mean;
      }
      if (mine && !bad && group.bad) report(p.status, EXTKV_DEV_BAD_NONPAD);
    }
  }
  __device__ __forceinline__ int64_t total() const { return __shfl_sync(0xffffffffu, end, 31); }
  // the cursor at the slice end that was cut at cell f (the warp's; f < total)
  __device__ __forceinline__ PrefixCursor<KT> cursor(const PrefixParams& p, const SliceAxis& axis, int64_t f) const {
    PrefixCursor<KT> c;
    c.g = __popc(__ballot_sync(0xffffffffu, end <= f));
    c.group.b0 = __shfl_sync(0xffffffffu, group.b0, c.g);
    c.group.rows = __shfl_sync(0xffffffffu, group.rows, c.g);
    c.group.lo = __shfl_sync(0xffffffffu, group.lo, c.g);
    c.group.hi = __shfl_sync(0xffffffffu, group.hi, c.g);
    c.group.bad = false;
    c.tiles = __shfl_sync(0xffffffffu, tiles, c.g);
    c.row_tiles = __shfl_sync(0xffffffffu, row_tiles, c.g);
    const int64_t units = static_cast<int64_t>(c.row_tiles) * p.Hkv;
    c.place(axis, mean, f - (__shfl_sync(0xffffffffu, end, c.g) - (c.tiles + cost_of(c.tiles, mean)) * units));
    return c;
  }
};

// The same for any number of groups, from scan_groups.
template <int KT, int NT>
__device__ __forceinline__ PrefixCursor<KT> prefix_cursor(const PrefixParams& p, const int64_t* pre, int per, const SliceAxis& axis,
                                                          int64_t mean, int64_t f) {
  int lo = 0, hi = NT;  // the last chunk whose first cell is <= f
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre[mid] <= f) lo = mid;
    else hi = mid;
  }
  PrefixCursor<KT> c;
  int64_t rest = f - pre[lo];
  for (c.g = lo * per;; ++c.g) {
    c.load(p);
    const int64_t n = cells_of_group<KT>(p, c.group, mean);
    if (rest < n) break;
    rest -= n;
  }
  c.place(axis, mean, rest);
  return c;
}

// A slice: the cursor at its start, and one behind it (g == G: behind all).
template <int KT>
struct Slice {
  PrefixCursor<KT> at;
  int end_g, end_u, end_t;
  __device__ __forceinline__ bool more(const PrefixParams& p) const {
    return at.g < end_g || (at.g == end_g && (at.u < end_u || (at.u == end_u && at.t < end_t)));
  }
  // tiles of the unit at hand that belong to the slice
  __device__ __forceinline__ int here() const { return at.g == end_g && at.u == end_u ? end_t - at.t : at.tiles - at.t; }
};
template <int KT, class F>  // F: the cursor at a cell
__device__ __forceinline__ Slice<KT> slice_of(const PrefixParams& p, const SliceAxis& axis, int i, F cursor) {
  Slice<KT> s;
  if (i >= axis.n) {  // none
    s.at.g = s.end_g = p.G;
    s.at.u = s.end_u = s.at.t = s.end_t = 0;
    return s;
  }
  s.at = cursor(axis.end(i));
  s.at.snap(p, axis);
  if (i + 1 < axis.n) {
    PrefixCursor<KT> e = cursor(axis.end(i + 1));
    e.snap(p, axis);
    s.end_g = e.g;
    s.end_u = e.u;
    s.end_t = e.t;
  } else {
    s.end_g = p.G;
    s.end_u = s.end_t = 0;
  }
  return s;
}

}  // namespace extkv
