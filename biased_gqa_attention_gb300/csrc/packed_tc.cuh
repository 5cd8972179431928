// packed_tc.cuh -- device parts shared by the tensor-core packed prefill kernels.
#pragma once

#include <climits>

#include "packed_plan.cuh"

namespace extkv {
namespace packed {

constexpr int kBM = 128;  // rows of a query tile
constexpr int kBN = 128;  // keys of a tile
constexpr uint32_t kWaitPolls = 1u << 22;
constexpr float kGrow = 8.f;  // log2 units

// Bounded wait that also gives up once another role has aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit) {
  if (limit > 0 && ptx::mbar_test_wait(bar, parity)) return true;  // cheaper than a suspending wait when it is there
  for (uint32_t i = 0; i < limit; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 127u) == 127u && *abort) return false;
  }
  *abort = 1;
  return false;
}

// One entry of the work list for one head group: two query tiles of
// tile_tok / 2 tokens each, or (split) one query tile twice, A with every other
// key tile and B with the rest.
struct Work {
  int row0, len, h0, hk;
  int tok[2];        // first token of query tiles A and B
  int lo[2], hi[2];  // their key tiles (of KN keys), every `step`-th (empty: tile B has no tokens, or no keys)
  int k_lo, k_hi;    // all key tiles
  int step;          // 1, or 2: split
  __device__ __forceinline__ bool joined() const { return step == 2 && lo[1] < hi[1]; }
};

template <int KN, bool SPLIT>
__device__ __forceinline__ Work work_at(const PackedParams& p, int64_t w) {
  Work r;
  const int64_t at = w / p.heads;
  const PackedItem it = p.items[item_in(p, at) ? at : 0];
  r.row0 = it.row0;
  r.len = it.len;
  r.h0 = static_cast<int>(w - at * p.heads) * p.pk;
  r.hk = r.h0 / p.g;
  const int tt = p.tile_tok / 2;
  r.k_lo = INT_MAX;
  r.k_hi = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int t0 = it.tok0 + (SPLIT && it.split ? 0 : t * tt), t1 = min(it.len, t0 + tt);
    r.tok[t] = t0;
    r.lo[t] = r.hi[t] = 0;
    if (t0 < t1) {
      r.lo[t] = (p.window > 0 ? max(0, t0 - p.window + 1) : 0) / KN;
      r.hi[t] = ((p.causal ? t1 : it.len) + KN - 1) / KN;
      r.k_lo = min(r.k_lo, r.lo[t]);
      r.k_hi = max(r.k_hi, r.hi[t]);
    }
  }
  r.step = SPLIT && it.split ? 2 : 1;
  if (r.step == 2) {
    const int n = r.k_hi - r.k_lo;
    r.lo[1] = r.k_lo + 1;
    r.hi[0] = r.k_lo + ((n - 1) | 1);       // behind A's last: tiles 0, 2, .. below n
    r.hi[1] = r.k_lo + (n / 2) * 2;         // behind B's last: tiles 1, 3, .. below n
    if (n < 2) r.lo[1] = r.hi[1] = 0;
  }
  return r;
}

// The work of worker `id` of `n`: rounds run over the list back and forth, so
// that a worker that got a dear item of one round gets a cheap one of the next.
struct Rounds {
  int64_t base = 0, n_work;
  int id, n, odd = 0;
  __device__ __forceinline__ Rounds(int64_t n_work_, int id_, int n_) : n_work(n_work_), id(id_), n(n_) {}
  // the next item, or -1
  __device__ __forceinline__ int64_t next() {
    const int64_t w = base + (odd ? n - 1 - id : id);
    base += n;
    odd ^= 1;
    return w < n_work ? w : -1;  // only the last round is short
  }
};

// One query row's scores over KN keys (raw q.k), in registers.
template <int KN>
struct Scores {
  static_assert(KN == 80 || KN == 128, "whole tensor-memory loads");
  static constexpr int Q = (KN + 31) / 32;
  uint32_t s[Q][32];
  __device__ __forceinline__ float at(int e) const { return __uint_as_float(s[e >> 5][e & 31]); }
  // from tensor memory at `ts`; keys outside [ra, rb) masked (k0: the first key)
  __device__ __forceinline__ void load(uint32_t ts) {
#pragma unroll
    for (int q = 0; q < KN / 32; ++q) ptx::tmem_ld32(ts + 32 * q, s[q]);
    if constexpr (KN % 32) ptx::tmem_ld16(ts + KN / 32 * 32, *reinterpret_cast<uint32_t(*)[16]>(s[Q - 1]));
    ptx::tmem_wait_ld();
  }
  __device__ __forceinline__ void mask(int ra, int rb, int k0) {
    if (__all_sync(0xffffffffu, ra <= k0 && rb >= k0 + KN)) return;
    const int a = ra - k0;
    const unsigned n = rb > ra ? rb - ra : 0;
#pragma unroll
    for (int e = 0; e < KN; ++e)
      if (static_cast<unsigned>(e - a) >= n) s[e >> 5][e & 31] = 0xff800000u;
  }
  __device__ __forceinline__ float max() const {
    float x[4] = {at(0), at(1), at(2), at(3)};
#pragma unroll
    for (int e = 4; e < KN; e += 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = e + 4 + i < KN ? ptx::max3(x[i], at(e + i), at(e + 4 + i)) : fmaxf(x[i], at(e + i));
    }
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  }
  // weights of keys E0 .. E0 + N - 1 against the maximum in nm = -m * c, as packed
  // bf16 (2^-8 of each weight off at most); ls sums them unrounded
  template <int E0, int N>
  __device__ __forceinline__ void weights(uint64_t c2, uint64_t nm2, uint64_t (&ls)[4], uint32_t (&pk)[N / 2]) const {
#pragma unroll
    for (int x = 0; x < N / 2; ++x) {
      const uint64_t d = ptx::fma2(ptx::f2(at(E0 + 2 * x), at(E0 + 2 * x + 1)), c2, nm2);
      const float e0 = ptx::ex2(ptx::f2_lo(d)), e1 = ptx::ex2(ptx::f2_hi(d));
      ls[x & 3] = ptx::add2(ls[x & 3], ptx::f2(e0, e1));
      pk[x] = ptx::pack_bf16x2(e0, e1);
    }
  }
};

// Takes the row's maximum over a new tile's scores `top` into m: lazily, when it
// has grown by more than kGrow, so that P stays below 2^8.  Then the row of O at
// `to` (D columns) and the sum l are rescaled, once `o_ready` says that the
// product that last wrote O is complete (false: that wait gave up, and so does
// this).
template <int D, class F>
__device__ __forceinline__ bool take_max(float top, uint32_t to, float c, float& m, float& l, F o_ready) {
  const float m_new = fmaxf(m, top);
  const bool grow = (m_new - m) * c > kGrow;  // false while the row has no key (NaN)
  const bool first = m == -INFINITY;
  if (__any_sync(0xffffffffu, grow && !first)) {
    if (!o_ready()) return false;
    const float f = grow && !first ? ptx::ex2((m - m_new) * c) : 1.f;
    l *= f;
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
      uint32_t o[32];
      ptx::tmem_ld32(to + 32 * q, o);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      ptx::tmem_st32(to + 32 * q, o);
    }
  }
  if (grow) m = m_new;
  return true;
}

// P written so far can be read by the tensor cores; then the warp together.
__device__ __forceinline__ void p_written() {
  ptx::tmem_wait_st();
  ptx::tc_fence_before();
  __syncwarp();
}

// One row of O at `to` over its sum l, into y (D columns) when `in`; `release`
// runs once the row has been read.
template <int D, class F>
__device__ __forceinline__ void store_row(uint32_t to, float l, bool in, __nv_bfloat16* y, F release) {
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    uint32_t o[2][32];
    ptx::tmem_ld32(to + 64 * q, o[0]);
    ptx::tmem_ld32(to + 64 * q + 32, o[1]);
    ptx::tmem_wait_ld();
    if (q == D / 64 - 1) release();
    if (in) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 8 * x + 2 * e;
          v[e] = ptx::pack_bf16x2(__uint_as_float(o[k >> 5][k & 31]) * inv, __uint_as_float(o[k >> 5][(k & 31) + 1]) * inv);
        }
        *reinterpret_cast<uint4*>(y + 64 * q + 8 * x) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

// The same for a row whose keys are in two parts: O at `ta` times fa and at `tb` times fb.
template <int D, class F>
__device__ __forceinline__ void store_joined(uint32_t ta, uint32_t tb, float fa, float fb, bool in, __nv_bfloat16* y,
                                             F release) {
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    uint32_t a[32], b[32];
    ptx::tmem_ld32(ta + 32 * q, a);
    ptx::tmem_ld32(tb + 32 * q, b);
    ptx::tmem_wait_ld();
    if (q == D / 32 - 1) release();
    if (in) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 8 * x + 2 * e;
          v[e] = ptx::pack_bf16x2(fmaf(__uint_as_float(b[k]), fb, __uint_as_float(a[k]) * fa),
                                  fmaf(__uint_as_float(b[k + 1]), fb, __uint_as_float(a[k + 1]) * fa));
        }
        *reinterpret_cast<uint4*>(y + 32 * q + 8 * x) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

// Zeroes V rows [r0, n) of a tile stored as 64-column chunks of n rows (128-byte
// swizzled rows; a whole row is zeroed, so the swizzle does not matter): rows
// behind a sequence's last have P = 0, but 0 * NaN would be NaN.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int n, int lane) {
  constexpr int kPieces = D / 8;  // 16 bytes each
  for (int x = r0 * kPieces + lane; x < n * kPieces; x += 32) {
    const int r = x / kPieces, ch = x % kPieces;
    *reinterpret_cast<uint4*>(tile + (ch >> 3) * (n * 128) + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  ptx::fence_proxy_async_smem();  // before the tensor cores read them
  __syncwarp();
}

}  // namespace packed
}  // namespace extkv
