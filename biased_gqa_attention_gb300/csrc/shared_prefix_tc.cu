// shared_prefix_tc.cu -- a shared prefix on the 5th-generation tensor cores: bf16,
// head sizes 64, 128 and 256, pages of whole boxes of 16 rows.
//
// Bound: a key of a KV head is 4 D bytes and 4 D flops a row, so with fewer rows than
// the card does flops a byte (285 at the measured rates) the prefix is bound by HBM,
// above that by the tensor pipe; a short one by the latency of its first and last steps.  A
// unit holds 256 rows (two M = 128 tiles A and B that share every K and V tile; one at
// head size 256, whose O takes half of tensor memory), so that the keys are read
// from memory once and from L2 once more for each 256 rows.
//   warp 0, 3     load K and V tiles of 64 keys into a ring of shared-memory units (TMA
//                 boxes of page rows, 128-byte swizzle), a lane per request
//   warp 1        loads Q (TMA boxes of a KV head's heads and several sequences), issues
//                 Q K^T of both row tiles
//   warp 2        issues P V of both
//   warps 4-7     tile A's rows: softmax, the partial result (and Q into shared memory where a
//                 row tile does not begin with a sequence)
//   warps 8-11    the same for tile B
// Rows are (sequence, query head) pairs, so a group may have any number of sequences and of
// heads.  Warps 0 to 3 find the CTA's slice of the axis of key tiles (SliceAxis) and hand
// it to the rows' warps; a unit's part in a CTA leaves (max, sum, O) in fp32.
//
// Registers (112 a thread at launch, from which the rows' warps take 128 and leave the
// others 72) and a ring of two K and two V tiles leave room on the SM for a CTA of the
// own pages' kernel (shared_prefix.cu), which runs beside this one.  64 sequences of 32 heads
// of 128 behind 8191 keys: 53 us the call, 74 where the kernels follow one another.  (Head size 64 has the
// same shares, although own pages follow it: with more registers a thread it was not measured.)
// Measured otherwise: tiles of 128 keys, with P over the S it is made from (both fill tensor
// memory), take 6000 clocks where two tiles of 64 take 3800, since each waits for the
// product before; one warp that issues everything 5000 (a product issued by a lane that the
// compiler does not know to be one alone takes 125 clocks to issue, see elect_one).
#include "packed_tc.cuh"
#include "shared_prefix.cuh"
#include "shared_prefix_tc.h"

#include <atomic>
#include <cstring>

namespace extkv {

namespace {

using namespace packed;

constexpr int kBarBytes = 1024;
constexpr int kTileKeys = 64;
constexpr int kSeen = 32;  // tiles whose pages' validity is kept: more than the ring holds

template <int D>
struct TcCfg {
  static constexpr int TILES = D == 256 ? 1 : 2;
  static constexpr int kThreads = TILES == 2 ? 384 : 256;
  static constexpr int KN = kTileKeys;
  static constexpr int kPart = KN / 2;  // keys of P released first
  static constexpr int kChunks = D / 64;
  // registers a thread at launch, and (two row tiles) of the warps that load and issue
  // and of those of the rows
  static constexpr int kRegs = TILES == 2 ? 112 : 240, kControlRegs = 72, kRowRegs = 128;
  static_assert(TILES == 1 || 4 * kControlRegs + 8 * kRowRegs <= 12 * kRegs, "shares of the launch's registers");
  static constexpr int kQTile = kBM * D * 2, kTile = KN * D * 2;
  static constexpr int kUnits = 4;  // K in the even ones, V in the odd ones
  static constexpr int kOffKV = TILES * kQTile;
  static constexpr int kOffBar = kOffKV + kUnits * kTile;
  static constexpr int kSmem = kOffBar + kBarBytes + 1024;
  // tensor memory of a tile: S, P, O
  static constexpr uint32_t kStride = TILES == 2 ? 256 : 512, kOCol = kStride - D;
  static constexpr uint32_t kPCol = KN;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, KN, 0, 0);
  static constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, D, 0, 1);
  static_assert(kPCol + KN / 2 <= kOCol, "tensor memory columns");
  static_assert(kSmem <= 232448 && kUnits / 2 + 2 <= kSeen, "shared memory");
  static_assert(kPart == 32, "a whole tensor-memory store");
};

struct TcBars {
  uint64_t q_full[2];
  uint64_t u_full[4], u_empty[4];
  uint64_t s_full[2], s_free[2], p_full[2][2], pv_done[2], o_full[2], o_free[2];
  uint64_t v_tail, drain[2];
  uint32_t boxes[kSeen];  // of each tile: which of its boxes lie in the pool
  uint32_t tmem_base;
  int abort;
  int64_t warp_sum[4];
  Slice<kTileKeys> slice;
};
static_assert(sizeof(TcBars) <= kBarBytes, "barrier block");

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A unit's part in this CTA: key tiles [t0, t1) of the slice's unit at hand.
template <int KN>
struct Segments {
  Slice<KN> s;
  int t0, t1;
  __device__ __forceinline__ Segments(const PrefixParams& p, const Slice<KN>& slice) : s(slice) { set(p); }
  __device__ __forceinline__ void set(const PrefixParams& p) {
    if (!more(p)) return;
    t0 = s.at.t;
    t1 = t0 + s.here();
  }
  __device__ __forceinline__ bool more(const PrefixParams& p) const { return s.more(p); }
  __device__ __forceinline__ void next(const PrefixParams& p) {
    s.at.t = t1 - 1;
    s.at.next(p);
    set(p);
  }
  __device__ __forceinline__ int rows(const PrefixParams& p, int t) const {  // of tile t
    return max(0, min(kBM, s.at.group.rows - s.at.row0(p) - t * kBM));
  }
};

template <int D>
__global__ void __maxnreg__(TcCfg<D>::kRegs)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PrefixParams p) {
  using C = TcCfg<D>;
  constexpr int KN = C::KN, TILES = C::TILES, NU = C::kUnits;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBars& bar = *reinterpret_cast<TcBars*>(sm + C::kOffBar);
  uint8_t* sKV = sm + C::kOffKV;
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;

  if (tid == 0) {
    for (int t = 0; t < TILES; ++t) {
      ptx::mbar_init(&bar.q_full[t], p.q_tma ? 1 : kBM);
      ptx::mbar_init(&bar.s_full[t], 1);
      ptx::mbar_init(&bar.s_free[t], 4);
      ptx::mbar_init(&bar.pv_done[t], 1);
      ptx::mbar_init(&bar.p_full[t][0], 4);
      ptx::mbar_init(&bar.p_full[t][1], 4);
      ptx::mbar_init(&bar.o_full[t], 1);
      ptx::mbar_init(&bar.o_free[t], kBM);
    }
    for (int u = 0; u < NU; ++u) {
      ptx::mbar_init(&bar.u_full[u], 1);
      ptx::mbar_init(&bar.u_empty[u], 1);
    }
    ptx::mbar_init(&bar.v_tail, 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&bar.drain[i], 1);
    bar.abort = 0;
    ptx::fence_mbar_init();
    if (p.q_tma) ptx::prefetch_tensormap(&qmap);
    ptx::prefetch_tensormap(&kmap);
    ptx::prefetch_tensormap(&vmap);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bar.tmem_base, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = bar.tmem_base;
  auto drain = [&](int who) {  // every product of an issuer has completed before tensor memory is released
    ptx::umma_commit(&bar.drain[who]);
    if (!ptx::mbar_wait_bounded(&bar.drain[who], 0, kWaitPolls)) *abort = 1;
  };

  if (warp < 4) {
    if constexpr (TILES == 2) reg_dec<C::kControlRegs>();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    // this CTA's slice of the axis; the scan's sums (more than 31 groups) lie where Q will
    constexpr int kFinders = 128;
    const bool few = p.G < 32;
    const GroupScan<KN> scan(p);
    int64_t* pre = reinterpret_cast<int64_t*>(sm);
    int per = 0;
    int64_t mean = scan.mean;
    if (!few) per = scan_groups<KN, kFinders, 1>(p, pre, bar.warp_sum, mean);
    const SliceAxis axis(p, few ? scan.total() : pre[kFinders], mean);
    const Slice<KN> slice = slice_of<KN>(p, axis, blockIdx.x, [&](int64_t f) {
      return few ? scan.cursor(p, axis, f) : prefix_cursor<KN, kFinders>(p, pre, per, axis, mean, f);
    });
    if (tid == 0) bar.slice = slice;
    if (!few) ptx::fence_proxy_async_smem();  // the sums' stores before Q's requests to the same place
    meet<2, C::kThreads>();  // the rows' warps have it; the sums have been read
    if (warp == 0 || warp == 3) {
      // ---------------- loads: K, and V by a warp of its own ----------------
      const bool is_v = warp == 3;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      const int boxes = KN / p.box, per_unit = boxes == 1 ? 1 : boxes * C::kChunks;  // requests of a tile
      const uint32_t all = (1u << boxes) - 1u;
      int u = is_v, tails = 0, seen = 0;
      bool ok = true;
      // the lane's request: a box of rows and (several boxes) one 64-column chunk of it
      const int my_box = boxes == 1 ? 0 : lane / C::kChunks, my_ch = boxes == 1 ? 0 : lane % C::kChunks;
      const int ahead = 32 / boxes;  // tiles whose pages the warp holds, a lane a box
      int first = 0, first_of = -1;  // the first key that some row of group first_of attends
      for (Segments<KN> s(p, slice); ok && s.more(p); s.next(p)) {
        const Group& g = s.s.at.group;
        const int hk = s.s.at.head(p);
        if (s.s.at.g != first_of) {
          first_of = s.s.at.g;
          first = first_of_group(p, g);
        }
        // the lane's box of the tiles from kt on: its first key, whether it is needed, and its page
        auto key = [&](int kt) { return (g.lo / KN + kt + lane / boxes) * KN + lane % boxes * p.box; };
        auto needed = [&](int kt) {
          const int j = key(kt);
          return lane < ahead * boxes && kt + lane / boxes < s.t1 && j < g.hi && j + p.box > first;
        };
        auto pages = [&](int kt) -> int64_t { return needed(kt) ? prefix_page(p, s.s.at.g, key(kt) / p.page_size) : -1; };
        int64_t page = pages(s.t0), next = pages(s.t0 + ahead);
        int window = s.t0;
        uint32_t in = 0;  // whose pages lie in the pool
        for (int kt = s.t0; kt < s.t1; ++kt, ++seen) {
          if (kt == s.t0 || kt == window + ahead) {
            if (kt != s.t0) {
              page = next;
              window = kt;
              next = pages(kt + ahead);
            }
            const bool good = page >= 0 && page < p.num_pages;
            if (!good && s.s.at.u == 0 && !is_v && needed(kt)) report(p.status, EXTKV_DEV_BAD_PAGE);
            in = __ballot_sync(0xffffffffu, good);
          }
          const int k0 = (g.lo / KN + kt) * KN, at = (kt - window) * boxes;
          const uint32_t mask = (in >> at) & all, bytes = __popc(mask) * p.box * D * 2;
          const int64_t my_page = __shfl_sync(0xffffffffu, page, at + my_box);
          const bool mine = lane < per_unit && ((mask >> my_box) & 1);
          const int off = (k0 + my_box * p.box) % p.page_size, row = static_cast<int>(my_page * p.Hkv + hk);
          // V: rows of keys that nobody attends become zeros, whatever they hold: their P is 0, and 0 * NaN would be NaN
          const bool ragged = is_v && (mask != all || k0 < first || k0 + KN > g.hi);
          if (!(ok = __all_sync(0xffffffffu, u < NU || wait_or_abort(&bar.u_empty[u % NU], ((u / NU) - 1) & 1, abort, lim)))) break;
          uint64_t* full = ragged ? &bar.v_tail : &bar.u_full[u % NU];
          uint8_t* dst = sKV + (u % NU) * C::kTile;
          if (lane == 0) {
            if (!is_v) bar.boxes[seen % kSeen] = mask;
            if (bytes) ptx::mbar_arrive_expect_tx(full, bytes);
            else ptx::mbar_arrive(full);
          }
          __syncwarp();
          if (mine) ptx::tma_load_4d(dst + my_ch * (KN * 128) + my_box * (p.box * 128), map, full, 0, off, row, my_ch);
          if (ragged) {
            if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.v_tail, tails & 1, abort, lim)))) break;
            ++tails;
            constexpr int kPieces = D / 8;
            const int r0 = mask == all && k0 >= first ? g.hi - k0 : 0;  // (only the prefix' end: from there)
            for (int x = r0 * kPieces + lane; x < KN * kPieces; x += 32) {
              const int r = x / kPieces, ch = x % kPieces, j = k0 + r;
              if (j < first || j >= g.hi || !((mask >> (r / p.box)) & 1))
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * (KN * 128) + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar.u_full[u % NU]);
          }
          u += 2;
        }
      }
      // Copies still in flight land before the CTA leaves, also where another warp gives
      // up only after this: the newest of each of this warp's units (a ragged V's have been
      // waited for, but where this warp gave up on them).
      if (lane == 0) {
        for (int x = max(u - NU, static_cast<int>(is_v)); x < u; x += 2) ptx::mbar_wait_bounded(&bar.u_full[x % NU], (x / NU) & 1, kWaitPolls >> 6);
        if (!ok && is_v) ptx::mbar_wait_bounded(&bar.v_tail, tails & 1, kWaitPolls >> 6);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- Q, Q K^T ----------------
      if (ptx::elect_one()) {
        const uint64_t qdesc = ptx::smem_desc_sw128(ptx::smem_u32(sm), 16, 1024);
        const uint64_t kdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, 1024);
        int u = 0;  // unit of the next K tile
        int nq[2] = {0, 0}, c[2] = {0, 0};  // a row tile's segments, products so far
        bool ok = true;
        for (Segments<KN> s(p, slice); ok && s.more(p); s.next(p)) {
          bool busy[2];
          for (int t = 0; t < 2; ++t) {
            busy[t] = t < TILES && s.rows(p, t) > 0;
            if (!ok || !busy[t]) continue;
            ++nq[t];
            if (p.q_tma) {  // once the products with the segment before's are complete
              if (c[t] > 0 && !(ok = wait_or_abort(&bar.s_full[t], (c[t] - 1) & 1, abort, lim))) continue;
              ptx::mbar_arrive_expect_tx(&bar.q_full[t], C::kQTile);
              ptx::tma_load_4d(sm + t * C::kQTile, &qmap, &bar.q_full[t], 0, s.s.at.head(p) * p.g,
                               s.s.at.group.b0 + (s.s.at.row0(p) + t * kBM) / p.g, 0);
            }
          }
          for (int kt = s.t0; ok && kt < s.t1; ++kt, u += 2) {
            if (!(ok = wait_or_abort(&bar.u_full[u % NU], (u / NU) & 1, abort, lim))) break;
            const uint64_t kd = kdesc + (((u % NU) * C::kTile) >> 4);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (!ok || !busy[t]) continue;
              if (kt == s.t0 && !(ok = wait_or_abort(&bar.q_full[t], (nq[t] - 1) & 1, abort, lim))) continue;
              // the scores before these are in the softmax's registers
              if (c[t] > 0 && !(ok = wait_or_abort(&bar.s_free[t], (c[t] - 1) & 1, abort, lim))) continue;
              ptx::tc_fence_after();
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                ptx::umma_bf16(tbase + t * C::kStride, qdesc + ((t * C::kQTile + (k >> 2) * (kBM * 128) + (k & 3) * 32) >> 4),
                               kd + (((k >> 2) * (KN * 128) + (k & 3) * 32) >> 4), C::kIdescQK, k > 0);
              ptx::umma_commit(&bar.s_full[t]);
              ++c[t];
            }
            if (ok) ptx::umma_commit(&bar.u_empty[u % NU]);
          }
        }
        if (slice.more(p)) drain(0);
        if (p.q_tma && !ok)  // copies in flight land before the CTA leaves
          for (int t = 0; t < TILES; ++t)
            if (nq[t]) ptx::mbar_wait_bounded(&bar.q_full[t], (nq[t] - 1) & 1, kWaitPolls >> 6);
      }
      __syncwarp();
    } else {
      // ---------------- P V ----------------
      if (ptx::elect_one()) {
        const uint64_t vdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), KN * 128, 1024);
        int u = 1;  // unit of the next V tile
        int nq[2] = {0, 0}, c[2] = {0, 0};  // a row tile's segments, products so far
        bool ok = true;
        for (Segments<KN> s(p, slice); ok && s.more(p); s.next(p)) {
          bool busy[2];
          for (int t = 0; t < 2; ++t) {
            busy[t] = t < TILES && s.rows(p, t) > 0;
            nq[t] += busy[t];
          }
          for (int kt = s.t0; ok && kt < s.t1; ++kt, u += 2) {
            if (!(ok = wait_or_abort(&bar.u_full[u % NU], (u / NU) & 1, abort, lim))) break;
            const bool first = kt == s.t0;
            const uint64_t vd = vdesc + (((u % NU) * C::kTile) >> 4);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (!ok || !busy[t]) continue;
              if (first && nq[t] > 1 && !(ok = wait_or_abort(&bar.o_free[t], (nq[t] - 2) & 1, abort, lim))) continue;
              const uint32_t tp = tbase + t * C::kStride + C::kPCol, to = tbase + t * C::kStride + C::kOCol;
#pragma unroll
              for (int k = 0; k < KN / 16; ++k) {
                if (ok && (k == 0 || k == C::kPart / 16)) {  // the first part of the keys while the others go through the softmax
                  ok = wait_or_abort(&bar.p_full[t][k > 0], c[t] & 1, abort, lim);
                  ptx::tc_fence_after();
                }
                if (ok) ptx::umma_bf16_ts(to, tp + k * 8, vd + ((k * 2048) >> 4), C::kIdescPV, (!first || k > 0) ? 1u : 0u);
              }
              if (!ok) continue;
              ptx::umma_commit(&bar.pv_done[t]);
              ++c[t];
              if (kt == s.t1 - 1) ptx::umma_commit(&bar.o_full[t]);
            }
            if (ok) ptx::umma_commit(&bar.u_empty[u % NU]);
          }
        }
        if (slice.more(p)) drain(1);
      }
      __syncwarp();
    }
  } else {
    // ---------------- rows: Q, softmax, partial results ----------------
    if constexpr (TILES == 2) reg_inc<C::kRowRegs>();
    meet<2, C::kThreads>();
    const Slice<KN> slice = bar.slice;
    const int t = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tbase + lane_base + t * C::kStride, tp = ts + C::kPCol, to = ts + C::kOCol;
    const float c = p.c;
    const uint64_t c2 = ptx::f2(c, c);
    const uint32_t all = KN / p.box == 32 ? ~0u : (1u << (KN / p.box)) - 1u;
    int nt = 0, no = 0, seen = 0;  // score tiles, segments with rows, tiles so far
    bool ok = true;
    for (Segments<KN> s(p, slice); ok && s.more(p); seen += s.t1 - s.t0, s.next(p)) {
      const bool whole = s.t0 == 0 && s.t1 == s.s.at.tiles;
      const int place = s.t0 == 0;
      const int rows = s.rows(p, t);
      if (rows == 0) continue;
      const Group& g = s.s.at.group;
      const int hk = s.s.at.head(p), in_unit = t * kBM + row, r = s.s.at.row0(p) + in_unit;
      const bool valid = row < rows;
      const int sq = valid ? r / p.g : 0, b = g.b0 + sq, h = hk * p.g + (valid ? r - sq * p.g : 0);
      // Q: the products with the segment before are complete, since its last scores have been read
      if (!p.q_tma) {
        const int64_t at = static_cast<int64_t>(b) * p.q_stride + static_cast<int64_t>(h) * D;
        const bool in = valid && EXTKV_IN_KIND(kChkRows, at, D, (p.B - 1) * p.q_stride + static_cast<int64_t>(p.Hq) * D, p.status);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at);
        uint8_t* dst = sm + t * C::kQTile + row * 128;
#pragma unroll
        for (int ch = 0; ch < C::kChunks; ++ch) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = in ? src[ch * 8 + i] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + ch * (kBM * 128) + ((i ^ (row & 7)) << 4)) = v[i];
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bar.q_full[t]);
      }
      // the row's keys [ra, rb)
      int ra = valid ? first_key(p, g.hi, own_length(p, b)) : 0, rb = g.hi;
      if (!valid) ra = rb = 0;
      float m = -INFINITY, l = 0.f;
      for (int kt = s.t0; kt < s.t1; ++kt, ++nt) {
        const int k0 = (g.lo / KN + kt) * KN;
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.s_full[t], nt & 1, abort, lim)))) break;
        ptx::tc_fence_after();
        Scores<KN> sc;
        sc.load(ts);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.s_free[t]);
        sc.mask(ra, rb, k0);
        const uint32_t have = bar.boxes[(seen + kt - s.t0) % kSeen];
        if (have != all) sc.mask_boxes(have, p.box);
        // PV(nt - 1) is complete: P may be written, O rescaled
        bool p_free = nt == 0;
        auto pv_complete = [&] {
          if (!p_free) {
            p_free = __all_sync(0xffffffffu, wait_or_abort(&bar.pv_done[t], (nt - 1) & 1, abort, lim));
            ptx::tc_fence_after();
          }
          return p_free;
        };
        if (!(ok = take_max<D>(sc.max(), to, c, m, l, pv_complete))) break;
        const float nm = m == -INFINITY ? 0.f : -m * c;
        const uint64_t nm2 = ptx::f2(nm, nm);
        uint64_t ls[4] = {0, 0, 0, 0};
        uint32_t pk[C::kPart / 2];
        sc.template weights<0, C::kPart>(c2, nm2, ls, pk);
        if (!(ok = pv_complete())) break;
        ptx::tmem_st16(tp, pk);
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[t][0]);
        uint32_t pk1[C::kPart / 2];
        sc.template weights<C::kPart, C::kPart>(c2, nm2, ls, pk1);
        ptx::tmem_st16(tp + C::kPart / 2, pk1);
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[t][1]);
        const uint64_t sum = ptx::add2(ptx::add2(ls[0], ls[1]), ptx::add2(ls[2], ls[3]));
        l += ptx::f2_lo(sum) + ptx::f2_hi(sum);
      }
      if (!ok) break;
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.o_full[t], no & 1, abort, lim)))) break;
      ++no;
      ptx::tc_fence_after();
      const int64_t at = whole ? static_cast<int64_t>(b) * p.Hq + h : (static_cast<int64_t>(blockIdx.x) * 2 + place) * p.rows + in_unit;
      const bool in = valid && (whole ? whole_in(p, at) : slice_in(p, at, 1));
      if (in) (whole ? p.whole_ml : p.ml)[at] = make_float2(m * c, l);
      float* dst = (whole ? p.whole : p.part) + at * D;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        ptx::tmem_ld32(to + 32 * q, o);
        ptx::tmem_wait_ld();
        if (in) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(dst + 32 * q + 4 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.o_free[t]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (tid == 0 && *abort) report(p.status, EXTKV_DEV_TIMEOUT);
  if (warp == 1) ptx::tmem_dealloc(tbase, C::kTmemCols);
}

template <int D>
cudaError_t launch(PrefixParams p, cudaStream_t s) {
  using C = TcCfg<D>;
  // (64 columns, row of a page, page and head, 64-column chunk)
  p.box = 16;
  while (p.box < C::KN && p.page_size % (2 * p.box) == 0) p.box *= 2;
  const bool one = p.box == C::KN;
  const uint64_t dims[4] = {64, static_cast<uint64_t>(p.page_size), static_cast<uint64_t>(p.num_pages) * p.Hkv, C::kChunks};
  const uint64_t str[3] = {D * 2, static_cast<uint64_t>(p.page_size) * D * 2, 128};
  const uint32_t box[4] = {64, static_cast<uint32_t>(p.box), 1, one ? static_cast<uint32_t>(C::kChunks) : 1u};
  CUtensorMap kmap, vmap, qmap;
  std::memset(&qmap, 0, sizeof qmap);
  if (!make_tensor_map_bf16(&kmap, p.k, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&vmap, p.v, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // q as (64 columns, head, sequence, 64-column chunk): a box is a row tile, where tiles begin with a sequence
  p.q_tma = kBM % p.g == 0;
  if (p.q_tma) {
    const uint64_t qdims[4] = {64, static_cast<uint64_t>(p.Hq), static_cast<uint64_t>(p.B), C::kChunks};
    const uint64_t qstr[3] = {D * 2, static_cast<uint64_t>(p.q_stride) * 2, 128};
    const uint32_t qbox[4] = {64, static_cast<uint32_t>(p.g), static_cast<uint32_t>(kBM / p.g), C::kChunks};
    if (!make_tensor_map_bf16(&qmap, p.q, 4, qdims, qstr, qbox, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  auto k = prefix_tc_kernel<D>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), C::kSmem); e != cudaSuccess) return e;
  if (C::TILES == 2) {  // the warps' shares of registers must fit what the launch gets, or they would wait for ever
    static std::atomic<int> regs{0};
    if (!regs) {
      cudaFuncAttributes a;
      if (cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(k)); e != cudaSuccess) return e;
      regs = a.numRegs;
    }
    if (4 * C::kControlRegs + 8 * C::kRowRegs > C::kThreads / 32 * regs) return cudaErrorLaunchOutOfResources;
  }
  PdlLaunch l(dim3(static_cast<unsigned>(p.slices)), C::kThreads, C::kSmem, s, C::TILES == 2);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, kmap, vmap, qmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool prefix_tc_supported(int64_t D, int dtype, int64_t page_size) {
  return dtype == EXTKV_BF16 && (D == 64 || D == 128 || D == 256) && page_size % 16 == 0 &&
         page_size * D * 2 < (int64_t(1) << 40);
}
int prefix_tc_rows(int64_t D) { return D == 256 ? kBM : 2 * kBM; }
int prefix_tc_tile_keys() { return kTileKeys; }

cudaError_t launch_prefix_tc(const PrefixParams& p, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, s) : p.D == 128 ? launch<128>(p, s) : launch<256>(p, s);
}

}  // namespace extkv
