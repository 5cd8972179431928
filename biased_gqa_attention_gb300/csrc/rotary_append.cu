// rotary_append.cu -- rotary positions with several axes, and the write of
// packed K/V rows into the cache's pages (rotated on the way).
//
// Both are HBM streams: every element is read once and written once.  A CTA
// takes a few rows: its threads first put the rows' angles (cos, sin per pair,
// shared by all heads of a row) and destinations into shared memory, then
// stream 16-byte vectors, a pair's two halves together.
//
// Angles.  Angle = position * inv_freq, up to 2^63 * 2^32 radians, of which
// only the fraction of a turn matters.  F = frac(inv_freq / 2 pi) as a 128-bit
// fixed-point number (inv_freq is 24 bits times a power of two, so this is one
// integer product with the first 96 bits of 1 / 2 pi); position * F wraps as
// angles wrap at a turn.  The upper 64 bits, a signed fraction, go to sincospif.
// Cut off are 2^-96 of a turn and less per radian (1 / 2 pi), less than 2^-128
// per position (F) and less than 2^-64 (the lower 64 bits).  No fp64.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace extkv {

namespace {

// Measured (GB300, the copy rate is 6.78 TB/s): 8194 rows of 24 heads of 256,
// 192 of each turned, 201 MB: 38 us, 5.3 TB/s; 8144 rows of q, K and V (32 + 2 +
// 2 heads of 128) into pages, 150 MB: 30 us, 5.0 TB/s.  One wave of CTAs beats
// more and smaller ones (4 rows a CTA: 36 us on the second), two vectors a
// thread with five CTAs beat four with four (41 us on the first), and
// prefetching the rows to L2 before the angles costs 3 us.
constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // rows per CTA
constexpr int kUnroll = 2;   // vectors in flight per thread
constexpr int kMinCtas = 5;
constexpr int kMaxHeadsPerCta = 4096;

struct Tensor {
  const void* src;
  void* dst;
  int64_t sb, ss, sh, db, ds, dh;
  int heads;
};

struct RotaryParams {
  Tensor q, k, v;
  int64_t S, n_rows;  // rows per batch, rows in all
  int D, R, n_axes;
  int sec_end[4];     // first pair past each axis
  const int64_t* positions;
  const float* inv_freq;
  int rows_per_cta, heads_per_cta;  // heads counted over q, k, v
  int64_t q_total, k_total;         // elements of q_out / k_out, and of the sources (checked builds)
  int64_t q_rows, k_rows, v_rows;
  int paged;
  const int64_t* page_table;
  const int64_t* write_idx;
  const int64_t* cu;
  int64_t n_seqs, num_pages, page_size, max_pages;
  int32_t* status;
};

// frac(f / 2 pi) * 2^128.  |f| = m * 2^e with a 24-bit m; 1 / 2 pi to 96 bits.
__device__ __forceinline__ unsigned __int128 turns_fixed(float f) {
  const uint32_t u = __float_as_uint(f) & 0x7fffffffu;
  const int ex = static_cast<int>(u >> 23);
  const uint32_t m = ex ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
  const uint64_t c_hi = 0x28BE60DBull, c_lo = 0x9391054A7F09D5F4ull;  // floor(2^96 / 2 pi)
  const unsigned __int128 p =
      static_cast<unsigned __int128>(c_lo) * m + (static_cast<unsigned __int128>(c_hi * m) << 64);
  const int sh = (ex ? ex : 1) - 150 + 32;  // e + 128 - 96
  return sh >= 0 ? p << sh : sh > -128 ? p >> -sh : 0;
}

// cos and sin of position * inv_freq
__device__ __forceinline__ float2 cos_sin(int64_t pos, float f) {
  if (!(fabsf(f) < 4294967296.f)) return make_float2(NAN, NAN);
  const unsigned __int128 F = turns_fixed(f);
  const uint64_t n = pos < 0 ? 0ull - static_cast<uint64_t>(pos) : static_cast<uint64_t>(pos);
  const uint64_t frac = static_cast<uint64_t>(F >> 64) * n + __umul64hi(static_cast<uint64_t>(F), n);
  float s, c;
  sincospif(static_cast<float>(static_cast<int64_t>(frac)) * 0x1p-63f, &s, &c);  // signed part of a turn
  return make_float2(c, (pos < 0) != (f < 0.f) ? -s : s);
}

template <typename T, int VW>
struct Vec;
template <typename T>
struct Vec<T, 1> {
  T v;
};
template <>
struct Vec<float, 4> {
  float4 v;
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 v;
};

template <typename T, int VW>
__device__ __forceinline__ void unpack(const Vec<T, VW>& x, float (&f)[VW]) {
  if constexpr (VW == 1) {
    f[0] = Elem<T>::to_float(x.v);
  } else if constexpr (sizeof(T) == 4) {
    f[0] = x.v.x;
    f[1] = x.v.y;
    f[2] = x.v.z;
    f[3] = x.v.w;
  } else {
    const uint32_t w[4] = {x.v.x, x.v.y, x.v.z, x.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int VW>
__device__ __forceinline__ void pack(Vec<T, VW>& x, const float (&f)[VW]) {
  if constexpr (VW == 1) {
    x.v = Elem<T>::from_float(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    x.v = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    x.v = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                     ptx::pack_bf16x2(f[6], f[7]));
  }
}

// x / d, exact while x * d < 2^32: a CTA divides (row, head) numbers, below
// kMaxRows * kMaxHeadsPerCta, by its heads.
static_assert(int64_t(kMaxRows) * kMaxHeadsPerCta * kMaxHeadsPerCta <= (int64_t(1) << 32), "SmallDiv");
struct SmallDiv {
  uint32_t d, inv;
  __device__ __forceinline__ explicit SmallDiv(int d_) : d(d_), inv(d_ > 1 ? 0xffffffffu / d_ + 1 : 0) {}
  __device__ __forceinline__ int operator()(int x) const { return d > 1 ? __umulhi(x, inv) : x; }
};

// Where a row goes; -1: nowhere.
struct RowPlace {
  int64_t q_src, q_dst, k_src, k_dst, v_src, v_dst;
};

// VW: elements per access (16 bytes, or 1 where a half of the rotated part is
// not whole vectors).  INTER: pairs (2i, 2i+1); else (i, i + R/2).
template <typename T, int VW, bool INTER>
__global__ void __launch_bounds__(kThreads, kMinCtas) rotary_append_kernel(const RotaryParams p) {
  extern __shared__ float2 cs[];  // [rows][PV][R/2 / PV]
  __shared__ RowPlace place[kMaxRows];
  const int tid = threadIdx.x;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.n_rows - row0));
  const int half = p.R / 2;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();

  // angle i of a vector's PV pairs, vector by vector, so that the threads of a
  // warp, which hold neighbouring vectors, read neighbouring words
  constexpr int PV = VW == 1 ? 1 : INTER ? VW / 2 : VW;
  const int n_vec = half / PV;
  for (int i = tid; i < rows * half; i += kThreads) {
    const int r = i / half, c = i - r * half;
    int axis = 0;
#pragma unroll
    for (int a = 0; a < 3; ++a) axis += c >= p.sec_end[a] ? 1 : 0;
    axis = min(axis, p.n_axes - 1);
    const int64_t pos_at = axis * p.n_rows + row0 + r;
    if (EXTKV_IN_KIND(kChkAngles, pos_at, 1, p.n_axes * p.n_rows, p.status) && EXTKV_IN_KIND(kChkAngles, c, 1, half, p.status))
      cs[r * half + (c % PV) * n_vec + c / PV] = cos_sin(p.positions[pos_at], p.inv_freq[c]);
  }
  if (tid >= kThreads - rows) {  // one of the last threads per row: its source and destination
    const int r = tid - (kThreads - rows);
    const int64_t t = row0 + r;
    RowPlace pl;
    if (!p.paged) {
      const int64_t b = t / p.S, s = t - b * p.S;
      pl.q_src = b * p.q.sb + s * p.q.ss;
      pl.q_dst = b * p.q.db + s * p.q.ds;
      pl.k_src = b * p.k.sb + s * p.k.ss;
      pl.k_dst = b * p.k.db + s * p.k.ds;
      pl.v_src = 0;
      pl.v_dst = -1;
    } else {
      int64_t b = t, first = t, end = t + 1;
      bool live = true;
      if (p.cu) {  // the last b with cu[b] <= t; a cu that is not ascending ends at some b, checked below
        int64_t lo = 0, hi = p.n_seqs + 1;
        while (lo < hi) {
          const int64_t mid = (lo + hi) >> 1;
          if (!EXTKV_IN_KIND(kChkLens, mid, 1, p.n_seqs + 1, p.status)) break;
          if (p.cu[mid] <= t) lo = mid + 1;
          else hi = mid;
        }
        b = lo - 1;
        live = b >= 0 && b < p.n_seqs;
        if (live && EXTKV_IN_KIND(kChkLens, b, 2, p.n_seqs + 1, p.status)) {
          first = p.cu[b];
          end = p.cu[b + 1];
          live = first >= 0 && first <= t && t < end && end <= p.n_rows;
        }
      }
      pl.q_src = t * p.q.ss;
      pl.q_dst = live ? t * p.q.ds : -1;
      pl.k_src = t * p.k.ss;
      pl.v_src = t * p.v.ss;
      pl.k_dst = pl.v_dst = -1;
      if (live && EXTKV_IN_KIND(kChkLens, b, 1, p.n_seqs, p.status)) {
        const int64_t w = p.write_idx[b], cap = p.max_pages * p.page_size;
        if (w < 0 || w > cap - (end - first)) {
          if (t == first && blockIdx.y == 0) report(p.status, EXTKV_DEV_BAD_WRITE_IDX);
        } else {
          const int64_t slot = w + (t - first), pg = slot / p.page_size;
          const int64_t at = b * p.max_pages + pg;
          const int64_t page = EXTKV_IN_KIND(kChkTable, at, 1, p.n_seqs * p.max_pages, p.status) ? p.page_table[at] : -1;
          if (page < 0 || page >= p.num_pages) {
            if (blockIdx.y == 0) report(p.status, EXTKV_DEV_BAD_PAGE);
          } else {
            pl.k_dst = pl.v_dst = (page * p.k.heads * p.page_size + (slot - pg * p.page_size)) * p.D;
          }
        }
      }
    }
    place[r] = pl;
  }
  if (p.cu && blockIdx.x == 0 && blockIdx.y == 0) {  // the whole of cu_seqlens, once
    bool bad = false;
    for (int64_t b = tid; b <= p.n_seqs; b += kThreads) {
      if (!EXTKV_IN_KIND(kChkLens, b, 1, p.n_seqs + 1, p.status)) break;
      const int64_t x = p.cu[b];
      bad |= x < 0 || x > p.n_rows || (b > 0 && p.cu[b - 1] > x);
    }
    if (bad) report(p.status, EXTKV_DEV_BAD_SEQLENS);
  }
  __syncthreads();

  const int h0 = blockIdx.y * p.heads_per_cta;
  const int h1 = min(h0 + p.heads_per_cta, p.q.heads + p.k.heads + p.v.heads);
  const int hv = p.q.heads + p.k.heads;  // first head of v
  using V = Vec<T, VW>;

  // q and k.  A thread keeps one place in the head (a pair of vectors to turn,
  // or a vector to copy) and walks over the CTA's (row, head)s, kUnroll at a time.
  const int rot = INTER && VW > 1 ? p.R / VW : half / VW;  // places that turn (single elements: R/2 pairs)
  const int per_head = rot + (p.D - p.R) / VW;
  const int nr = max(0, min(h1, hv) - h0);
  const SmallDiv by_nr(nr);
  for (int c0 = 0; c0 < per_head; c0 += kThreads) {  // once, but for single elements of wide heads
    const int here = min(per_head - c0, kThreads), step = kThreads / here;
    const int lane_h = tid / here, c = c0 + tid - lane_h * here;
    const int total = lane_h < step ? rows * nr : 0;
    const bool turn = c < rot;
    const int e = !turn ? p.R + (c - rot) * VW : INTER && VW == 1 ? 2 * c : c * VW;  // first element
    const int part = turn && !(INTER && VW > 1) ? (INTER ? 1 : half) : 0;           // distance of the pair's other vector
    for (int x0 = lane_h; x0 < total; x0 += step * kUnroll) {
      const T* src[kUnroll];
      T* dst[kUnroll];
      int row[kUnroll];
      V a[kUnroll], b[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int x = x0 + u * step;
        src[u] = nullptr;
        if (x < total) {
          const int r = by_nr(x), h = h0 + x - r * nr;
          const bool is_q = h < p.q.heads;
          const Tensor& t = is_q ? p.q : p.k;
          const int hd = is_q ? h : h - p.q.heads;
          const int64_t to = is_q ? place[r].q_dst : place[r].k_dst;
          const int64_t d_at = to + hd * t.dh + e, s_at = (is_q ? place[r].q_src : place[r].k_src) + hd * t.sh + e;
          if (to >= 0 &&
              EXTKV_IN_KIND(is_q || !p.paged ? kChkOut : kChkPages, d_at, part + VW, is_q ? p.q_total : p.k_total, p.status) &&
              EXTKV_IN_KIND(kChkRows, s_at, part + VW, is_q ? p.q_rows : p.k_rows, p.status)) {
            src[u] = static_cast<const T*>(t.src) + s_at;
            dst[u] = static_cast<T*>(t.dst) + d_at;
            row[u] = r;
            a[u] = *reinterpret_cast<const V*>(src[u]);
            if (part) b[u] = *reinterpret_cast<const V*>(src[u] + part);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (!src[u]) continue;
        if (turn) {
          const float2* w = cs + row[u] * half + c;
          float f[VW], g[VW];
          unpack<T, VW>(a[u], f);
          if (INTER && VW > 1) {
#pragma unroll
            for (int i = 0; i + 1 < VW; i += 2) {
              const float2 q = w[(i / 2) * n_vec];
              const float x = f[i], y = f[i + 1];
              f[i] = x * q.x - y * q.y;
              f[i + 1] = y * q.x + x * q.y;
            }
          } else {
            unpack<T, VW>(b[u], g);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
              const float2 q = w[i * n_vec];
              const float x = f[i], y = g[i];
              f[i] = x * q.x - y * q.y;
              g[i] = y * q.x + x * q.y;
            }
            pack<T, VW>(b[u], g);
          }
          pack<T, VW>(a[u], f);
        }
        *reinterpret_cast<V*>(dst[u]) = a[u];
        if (part) *reinterpret_cast<V*>(dst[u] + part) = b[u];
      }
    }
  }

  // v: copies of whole heads, 16 bytes at a time (D is whole vectors)
  constexpr int CW = 16 / sizeof(T);
  const int nv = max(0, h1 - max(h0, hv)), hv0 = max(h0, hv) - hv, per_v = p.D / CW;
  const int step = kThreads / per_v, lane_h = tid / per_v, e = (tid - lane_h * per_v) * CW;
  const int total = lane_h < step ? rows * nv : 0;
  const SmallDiv by_nv(nv);
  for (int x0 = lane_h; x0 < total; x0 += step * kUnroll) {
    uint4 a[kUnroll];
    T* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = x0 + u * step;
      dst[u] = nullptr;
      if (x < total) {
        const int r = by_nv(x), hd = hv0 + x - r * nv;
        const int64_t d_at = place[r].v_dst + hd * p.v.dh + e, s_at = place[r].v_src + hd * p.v.sh + e;
        if (place[r].v_dst >= 0 && EXTKV_IN_KIND(kChkPages, d_at, CW, p.k_total, p.status) &&
            EXTKV_IN_KIND(kChkRows, s_at, CW, p.v_rows, p.status)) {
          dst[u] = static_cast<T*>(p.v.dst) + d_at;
          a[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v.src) + s_at);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = a[u];
  }
}

Tensor to_tensor(const RowTensor& t) { return Tensor{t.src, t.dst, t.sb, t.ss, t.sh, t.db, t.ds, t.dh, t.heads}; }

template <typename T>
cudaError_t launch_typed(const RotaryArgs& a, const RotaryParams& p, dim3 grid, size_t smem) {
  constexpr int kVW = 16 / sizeof(T);
  const bool inter = a.rotary && a.rotary->interleaved;
  // whole vectors: both halves of the rotated part (interleaved: the part) start on one
  const bool wide = inter ? p.R % kVW == 0 : (p.R / 2) % kVW == 0;
  PdlLaunch l(grid, kThreads, smem, a.stream);
  cudaError_t e;
  if (inter)
    e = wide ? cudaLaunchKernelEx(&l.cfg, rotary_append_kernel<T, kVW, true>, p)
             : cudaLaunchKernelEx(&l.cfg, rotary_append_kernel<T, 1, true>, p);
  else
    e = wide ? cudaLaunchKernelEx(&l.cfg, rotary_append_kernel<T, kVW, false>, p)
             : cudaLaunchKernelEx(&l.cfg, rotary_append_kernel<T, 1, false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a) {
  RotaryParams p{};
  p.q = to_tensor(a.q);
  p.k = to_tensor(a.k);
  p.v = to_tensor(a.v);
  p.S = a.S;
  p.n_rows = a.B * a.S;
  p.D = static_cast<int>(a.D);
  if (a.rotary) {
    p.R = a.rotary->rotary_dim;
    p.n_axes = a.rotary->n_axes;
    int end = 0;
    for (int i = 0; i < 4; ++i) {
      if (i < p.n_axes) end += a.rotary->sections[i];
      p.sec_end[i] = end;
    }
    p.positions = a.rotary->positions;
    p.inv_freq = a.rotary->inv_freq;
  }
  p.q_total = p.n_rows * a.q.heads * a.D;
  p.k_total = a.paged ? a.num_pages * a.page_size * a.k.heads * a.D : p.n_rows * a.k.heads * a.D;
  // (sources: dense batches, or the rows of a packed tensor)
  auto elements = [&](const RowTensor& t) {
    return t.heads ? (a.B - 1) * t.sb + (a.S - 1) * t.ss + (t.heads - 1) * t.sh + a.D : 0;
  };
  p.q_rows = elements(a.q);
  p.k_rows = elements(a.k);
  p.v_rows = elements(a.v);
  p.paged = a.paged;
  p.page_table = a.page_table;
  p.write_idx = a.write_idx;
  p.cu = a.cu_seqlens;
  p.n_seqs = a.n_seqs;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.status = a.status;
  // Few rows: a CTA per row and per some of its heads, so that a decode step's
  // few hundred kilobytes spread over the GPU (each CTA computes its row's
  // angles again), as long as they make one wave: 300 rows of 10 heads of 128 take
  // 8 us so, 10 with CTAs for more than one wave, 50 rows of 72 heads of 256 8 and 10.
  // Many rows: as many rows a CTA as make one wave of CTAs.
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  const int64_t ctas = int64_t(num_sms()) * kMinCtas;
  int hpc = std::min(heads, kMaxHeadsPerCta);
  while (hpc > 4 && 2 * p.n_rows * ((heads + hpc - 1) / hpc) <= ctas) hpc = (hpc + 1) / 2;
  const int64_t rpc = hpc == heads ? std::min<int64_t>(kMaxRows, (p.n_rows + ctas - 1) / ctas) : 1;
  const int64_t gx = (p.n_rows + rpc - 1) / rpc;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  p.rows_per_cta = static_cast<int>(rpc);
  p.heads_per_cta = hpc;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((heads + hpc - 1) / hpc));
  const size_t smem = rpc * (p.R / 2) * sizeof(float2);
  return a.dtype == EXTKV_F32 ? launch_typed<float>(a, p, grid, smem) : launch_typed<__nv_bfloat16>(a, p, grid, smem);
}

}  // namespace extkv
