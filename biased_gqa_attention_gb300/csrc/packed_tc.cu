// packed_tc.cu -- packed prefill on the 5th-generation tensor cores: bf16, head
// sizes 64 and 128.
//
// Bound: the tensor pipe for long prompts (4 D flops a pair against one
// exponential a pair), the softmax's instruction rate close behind it.
//
// A persistent CTA per SM takes query tiles from the plan's list (dearest
// first, rounds taken in alternating order).  An item is 256 query rows, two
// M = 128 tiles A and B of one KV head's (token, head) rows; or, where one item
// would outlast a CTA's share of the batch, 128 rows: then A takes its first, third, ..
// key tile and B the others, and A's softmax warps join the two, B's rows of O
// straight from tensor memory.
//   warp 0       loads: Q tiles, then K and V tiles of KN keys through a ring of
//                shared-memory units (TMA, 128-byte swizzle)
//   warps 1, 2   issue Q K^T of tile A and of tile B
//   warps 4, 5   issue P V of tile A and of tile B
//   warps 8-11   softmax and output of tile A, a query row per thread
//   warps 12-15  the same for tile B
// (warps 3, 6 and 7 only fill warpgroups: the first two give registers to the
// softmax's.)
// Tensor memory holds S, P (bf16) and O of each tile apart from each other, so
// the two products of a tile depend on each other only through the softmax:
// QK(j + 1) is issued as soon as the softmax has S(j) in registers and runs
// beside it.  That is what fixes KN at head size 128: 80 + 40 + 128 columns, of
// 256 a tile.  Four issuers, because a thread's barrier tests (some hundred
// cycles each) stand between its products, and the pipe empties meanwhile:
// measured alone it takes one 128 x 128 x 16 MMA every 64 cycles from one thread.
// A 16001-token prompt of 8 heads of 128: 515 us with one issuer and P over an S
// of 128 keys, 462 us with one per tile, 486 us with S and P apart, 391 us so
// (1340 TFLOP/s, 0.70 of the measured cuBLAS rate).
#include "internal.h"
#include "packed_tc.cuh"
#include "packed_tc.h"
#include "tma_host.h"

namespace extkv {

namespace {

using namespace packed;

constexpr int kMaxUnits = 8;

// barriers, then B's (max, sum) of each row for the join
constexpr int kBarBytes = 512, kJoinBytes = kBM * 8;

template <int D>
struct Cfg {
  static constexpr int kThreads = 512;
  static constexpr int KN = D == 64 ? 128 : 80;  // keys of a tile
  static constexpr int kPart = D == 64 ? 64 : 48;  // keys of P released first
  static constexpr int kQTile = kBM * D * 2, kTile = KN * D * 2;  // bytes of a Q and of a K or V tile
  static constexpr int kFit = (232448 - 1024 - kBarBytes - kJoinBytes - 2 * kQTile) / kTile;
  static constexpr int kUnits = kFit < kMaxUnits ? kFit : kMaxUnits;
  static constexpr int kOffKV = 2 * kQTile;
  static constexpr int kOffBar = kOffKV + kUnits * kTile;
  static constexpr int kSmem = kOffBar + kBarBytes + kJoinBytes + 1024;
  // tensor memory of a tile: S, P, O
  static constexpr uint32_t kStride = 256, kPCol = KN, kOCol = kStride - D;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, KN, 0, 0);
  static_assert(kPCol + KN / 2 <= kOCol, "tensor memory columns");
  // K units keep to the even slots and V units to the odd ones, so that the
  // warps that read only the ones or the others see every phase of their slots
  static_assert(kUnits % 2 == 0, "ring");
  static constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, D, 0, 1);
  static_assert(kSmem <= 232448 && kUnits >= 4, "shared memory");
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t u_full[kMaxUnits], u_empty[kMaxUnits];
  uint64_t s_full[2], s_free[2], p_full[2][2], pv_done[2], o_full[2], o_free[2];  // p_full: of each part of P
  uint64_t v_tail, drain[4], join;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

// Registers of the calling warpgroup; 256 * 72 + 256 * 176 <= 512 * 128.
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// SPLIT: the list may hold split items (the case above, which has none: 391 us
// without and 398 with).
template <int D, bool SPLIT>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const PackedParams p) {
  using C = Cfg<D>;
  constexpr int KN = C::KN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(sm + C::kOffBar);
  uint8_t* sKV = sm + C::kOffKV;
  float2* join_ml = reinterpret_cast<float2*>(sm + C::kOffBar + kBarBytes);
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&bar.q_full[t], 1);
      ptx::mbar_init(&bar.q_empty[t], 1);
      ptx::mbar_init(&bar.s_full[t], 1);
      ptx::mbar_init(&bar.s_free[t], 4);
      ptx::mbar_init(&bar.pv_done[t], 1);
      ptx::mbar_init(&bar.p_full[t][0], 4);
      ptx::mbar_init(&bar.p_full[t][1], 4);
      ptx::mbar_init(&bar.o_full[t], 1);
      ptx::mbar_init(&bar.o_free[t], 128);
    }
    for (int u = 0; u < C::kUnits; ++u) {
      ptx::mbar_init(&bar.u_full[u], 1);
      ptx::mbar_init(&bar.u_empty[u], 2);
    }
    ptx::mbar_init(&bar.v_tail, 1);
    ptx::mbar_init(&bar.join, 128);
    for (int t = 0; t < 4; ++t) ptx::mbar_init(&bar.drain[t], 1);
    bar.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tensormap(&qmap);
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
  ptx::grid_dependency_wait();  // the plan, and what the caller ran before it
  const int64_t n_work = static_cast<int64_t>(*p.count) * p.heads;

  // every MMA an issuer issued has completed before tensor memory is released
  auto drain = [&](bool issued, int who) {
    if (!issued) return;
    ptx::umma_commit(&bar.drain[who - 1]);
    if (!ptx::mbar_wait_bounded(&bar.drain[who - 1], 0, kWaitPolls)) *abort = 1;
  };

  if (warp < 8) {
    reg_dec<72>();
    if (warp == 0) {
      // ---------------- loads ----------------
      int u = 0, nq[2] = {0, 0}, tails = 0;
      bool ok = true;
      auto acquire = [&]() -> bool {  // the next unit of the ring is free
        return u < C::kUnits || wait_or_abort(&bar.u_empty[u % C::kUnits], ((u / C::kUnits) - 1) & 1, abort, lim);
      };
      auto load_q = [&](const Work& w, int t) -> bool {
        if (w.lo[t] >= w.hi[t]) return true;
        if (nq[t] && !wait_or_abort(&bar.q_empty[t], (nq[t] - 1) & 1, abort, lim)) return false;
        ptx::mbar_arrive_expect_tx(&bar.q_full[t], C::kQTile);
        ptx::tma_load_4d(sm + t * C::kQTile, &qmap, &bar.q_full[t], 0, w.h0, w.row0 + (t ? w.tok[1] : w.tok[0]), 0);
        ++nq[t];
        return true;
      };
      Rounds rounds(n_work, blockIdx.x, gridDim.x);
      for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
        const Work w = work_at<KN, SPLIT>(p, wi);
        if (lane == 0) ok = load_q(w, 0);
        for (int kt = w.k_lo; kt < w.k_hi; ++kt) {
          const int key0 = w.row0 + kt * KN;
          const bool tail = (kt + 1) * KN > w.len;  // keys of the next sequence behind the last one
          if (lane == 0) {
            ok = ok && acquire();
            if (ok) {
              uint64_t* full = &bar.u_full[u % C::kUnits];
              ptx::mbar_arrive_expect_tx(full, C::kTile);
              ptx::tma_load_4d(sKV + (u % C::kUnits) * C::kTile, &kmap, full, 0, key0, w.hk, 0);
            }
            if (ok && kt == w.k_lo) ok = load_q(w, 1);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          ++u;
          uint8_t* dst = sKV + (u % C::kUnits) * C::kTile;
          if (lane == 0) {
            ok = acquire();
            if (ok) {
              uint64_t* full = tail ? &bar.v_tail : &bar.u_full[u % C::kUnits];
              ptx::mbar_arrive_expect_tx(full, C::kTile);
              ptx::tma_load_4d(dst, &vmap, full, 0, key0, w.hk, 0);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (tail) {
            if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.v_tail, tails & 1, abort, lim)))) break;
            ++tails;
            zero_rows<D>(dst, w.len - kt * KN, KN, lane);
            if (lane == 0) ptx::mbar_arrive(&bar.u_full[u % C::kUnits]);
          }
          ++u;
        }
      }
      // Copies still in flight land before the CTA leaves, also where another warp
      // gives up only after this: the newest of each slot and of Q, and where
      // this warp gave up the unit it stood at, which may have been sent.
      if (lane == 0) {
        const int sent = ok ? u : u + 1;
        for (int x = sent > C::kUnits ? sent - C::kUnits : 0; x < sent; ++x)
          ptx::mbar_wait_bounded(&bar.u_full[x % C::kUnits], (x / C::kUnits) & 1, kWaitPolls >> 6);
        for (int t = 0; t < 2; ++t)
          if (nq[t]) ptx::mbar_wait_bounded(&bar.q_full[t], (nq[t] - 1) & 1, kWaitPolls >> 6);
        if (!ok) ptx::mbar_wait_bounded(&bar.v_tail, tails & 1, kWaitPolls >> 6);
      }
      __syncwarp();
    } else if (warp < 3) {
      // ---------------- Q K^T of one query tile ----------------
      if (lane == 0) {
        const int t = warp - 1;
        const uint64_t qdesc = ptx::smem_desc_sw128(ptx::smem_u32(sm + t * C::kQTile), 16, 1024);
        const uint64_t kdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, 1024);
        const uint32_t ts = tbase + t * C::kStride;
        int u = 0, nq = 0, c = 0;  // unit of the next K tile, items, products so far
        bool ok = true, issued = false;
        Rounds rounds(n_work, blockIdx.x, gridDim.x);
        for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
          const Work w = work_at<KN, SPLIT>(p, wi);
          const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
          issued = true;
          nq += lo < hi;
          for (int kt = w.k_lo; kt < w.k_hi; ++kt, u += 2) {
            if (!(ok = wait_or_abort(&bar.u_full[u % C::kUnits], (u / C::kUnits) & 1, abort, lim))) break;
            if (kt >= lo && kt < hi && (!SPLIT || ((kt - lo) & (w.step - 1)) == 0)) {
              if (kt == lo && !(ok = wait_or_abort(&bar.q_full[t], (nq - 1) & 1, abort, lim))) break;
              // the scores before these are in the softmax's registers
              if (c > 0 && !(ok = wait_or_abort(&bar.s_free[t], (c - 1) & 1, abort, lim))) break;
              ptx::tc_fence_after();
              const uint64_t kd = kdesc + (((u % C::kUnits) * C::kTile) >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                ptx::umma_bf16(ts, qdesc + (((k >> 2) * (kBM * 128) + (k & 3) * 32) >> 4),
                               kd + (((k >> 2) * (KN * 128) + (k & 3) * 32) >> 4), C::kIdescQK, k > 0);
              ptx::umma_commit(&bar.s_full[t]);
              ++c;
              if (kt == hi - 1) ptx::umma_commit(&bar.q_empty[t]);
            }
            ptx::umma_commit(&bar.u_empty[u % C::kUnits]);
          }
        }
        drain(issued, warp);
      }
      __syncwarp();
    } else if (warp == 4 || warp == 5) {
      // ---------------- P V of one query tile ----------------
      if (lane == 0) {
        const int t = warp - 4;
        const uint64_t vdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), KN * 128, 1024);
        const uint32_t tp = tbase + t * C::kStride + C::kPCol, to = tbase + t * C::kStride + C::kOCol;
        int u = 1, nq = 0, c = 0;  // unit of the next V tile, items, products so far
        bool ok = true, issued = false;
        Rounds rounds(n_work, blockIdx.x, gridDim.x);
        for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
          const Work w = work_at<KN, SPLIT>(p, wi);
          const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
          issued = true;
          nq += lo < hi;
          for (int kt = w.k_lo; kt < w.k_hi && ok; ++kt, u += 2) {
            if (!(ok = wait_or_abort(&bar.u_full[u % C::kUnits], (u / C::kUnits) & 1, abort, lim))) break;
            if (kt >= lo && kt < hi && (!SPLIT || ((kt - lo) & (w.step - 1)) == 0)) {
              const bool first = kt == lo;
              if (first && nq > 1 && !(ok = wait_or_abort(&bar.o_free[t], (nq - 2) & 1, abort, lim))) break;
              const uint64_t vd = vdesc + (((u % C::kUnits) * C::kTile) >> 4);
#pragma unroll
              for (int k = 0; k < KN / 16; ++k) {
                // the first part of the keys while the others go through the softmax
                if (k == 0 || k == C::kPart / 16) {
                  if (!(ok = wait_or_abort(&bar.p_full[t][k > 0], c & 1, abort, lim))) break;
                  ptx::tc_fence_after();
                }
                ptx::umma_bf16_ts(to, tp + k * 8, vd + ((k * 2048) >> 4), C::kIdescPV, (!first || k > 0) ? 1u : 0u);
              }
              if (!ok) break;
              ptx::umma_commit(&bar.pv_done[t]);
              ++c;
              if (kt == hi - 1) ptx::umma_commit(&bar.o_full[t]);
            }
            ptx::umma_commit(&bar.u_empty[u % C::kUnits]);
          }
        }
        drain(issued, warp - 1);
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax and output ----------------
    reg_inc<176>();
    const int t = (warp - 8) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tbase + lane_base + t * C::kStride, tp = ts + C::kPCol, to = ts + C::kOCol;
    const float c = p.c;
    const uint64_t c2 = ptx::f2(c, c);
    int n = 0, no = 0, nb = 0, nj = 0;  // score tiles, items, B's items and joins so far
    bool ok = true;
    Rounds rounds(n_work, blockIdx.x, gridDim.x);
    for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
      const Work w = work_at<KN, SPLIT>(p, wi);
      const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
      if (lo >= hi) continue;
      const int tok = (t ? w.tok[1] : w.tok[0]) + row / p.pk;
      // the row's keys [ra, rb)
      int ra = p.window > 0 ? max(0, tok - p.window + 1) : 0, rb = p.causal ? tok + 1 : w.len;
      const bool valid = tok < w.len;
      if (!valid) ra = rb = 0;
      float m = -INFINITY, l = 0.f;
      for (int kt = lo; kt < hi; kt += SPLIT ? w.step : 1, ++n) {
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.s_full[t], n & 1, abort, lim)))) break;
        ptx::tc_fence_after();
        Scores<KN> s;
        s.load(ts);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.s_free[t]);
        s.mask(ra, rb, kt * KN);
        // PV(n - 1) is complete: P may be written, O rescaled
        bool p_free = n == 0;
        auto pv_complete = [&] {
          if (!p_free) {
            p_free = __all_sync(0xffffffffu, wait_or_abort(&bar.pv_done[t], (n - 1) & 1, abort, lim));
            ptx::tc_fence_after();
          }
          return p_free;
        };
        if (!(ok = take_max<D>(s.max(), to, c, m, l, pv_complete))) break;
        const float nm = m == -INFINITY ? 0.f : -m * c;
        const uint64_t nm2 = ptx::f2(nm, nm);
        uint64_t ls[4] = {0, 0, 0, 0};
        uint32_t pk[C::kPart / 2];
        s.template weights<0, C::kPart>(c2, nm2, ls, pk);
        if (!(ok = pv_complete())) break;
        if constexpr (C::kPart == 64) {
          ptx::tmem_st32(tp, pk);
        } else {
          ptx::tmem_st16(tp, *reinterpret_cast<uint32_t(*)[16]>(pk));
          ptx::tmem_st8(tp + 16, *reinterpret_cast<uint32_t(*)[8]>(pk + 16));
        }
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[t][0]);
        uint32_t pk1[(KN - C::kPart) / 2];
        s.template weights<C::kPart, KN - C::kPart>(c2, nm2, ls, pk1);
        if constexpr (KN - C::kPart == 64) ptx::tmem_st32(tp + C::kPart / 2, pk1);
        else ptx::tmem_st16(tp + C::kPart / 2, pk1);
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[t][1]);
        const uint64_t sum = ptx::add2(ptx::add2(ls[0], ls[1]), ptx::add2(ls[2], ls[3]));
        l += ptx::f2_lo(sum) + ptx::f2_hi(sum);
      }
      if (!ok) break;
      const bool joined = SPLIT && w.joined();
      if (joined && t == 1) {
        // the rows' maxima and sums to A's warps, which read O: once they have
        // read those of this tile's item before (an item of its own passes at once)
        if (no > 0 && !(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.o_free[1], (no - 1) & 1, abort, lim)))) break;
        ++no;
        join_ml[row] = make_float2(m, l);
        ptx::mbar_arrive(&bar.join);
        continue;
      }
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.o_full[t], no & 1, abort, lim)))) break;
      ++no;
      if (joined) {
        // B's sums first: then B has left its item before, and the phase of its
        // o_full that is waited for is the next to complete
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.join, nj & 1, abort, lim) &&
                                               wait_or_abort(&bar.o_full[1], nb & 1, abort, lim))))
          break;
        ++nj;
      }
      nb += w.lo[1] < w.hi[1];
      ptx::tc_fence_after();
      const int64_t y0 = (static_cast<int64_t>(w.row0 + tok) * p.Hq + w.h0 + row % p.pk) * D;
      const bool in = valid && EXTKV_IN_KIND(kChkOut, y0, D, static_cast<int64_t>(p.T) * p.Hq * D, p.status);
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + y0;
      if (joined) {
        const float2 o = join_ml[row];
        const float mm = fmaxf(m, o.x), ref = mm == -INFINITY ? 0.f : mm;
        const float fa = m == -INFINITY ? 0.f : ptx::ex2((m - ref) * c), fb = o.x == -INFINITY ? 0.f : ptx::ex2((o.x - ref) * c);
        const float sum = fmaf(l, fa, o.y * fb), inv = sum != 0.f ? 1.f / sum : 0.f;
        store_joined<D>(to, to + C::kStride, fa * inv, fb * inv, in, y, [&] {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&bar.o_free[0]);
          ptx::mbar_arrive(&bar.o_free[1]);
        });
      } else {
        store_row<D>(to, l, in, y, [&] {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&bar.o_free[t]);
        });
      }
    }
  }
  ptx::grid_launch_dependents();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (tid == 0 && *abort) report(p.status, EXTKV_DEV_TIMEOUT);
  if (warp == 1) ptx::tmem_dealloc(tbase, C::kTmemCols);
}

template <int D>
cudaError_t launch(const PackedParams& p, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap qmap, kmap, vmap;
  const uint64_t T = p.T, chunks = D / 64;
  const uint32_t tt = p.tile_tok / 2;
  // (64 columns, head, row, 64-column chunk): a box lands a tile's (token, head)
  // rows one after another
  const uint64_t q_dims[4] = {64, static_cast<uint64_t>(p.Hq), T, chunks};
  const uint64_t q_str[3] = {D * 2, static_cast<uint64_t>(p.q_stride) * 2, 128};
  const uint32_t q_box[4] = {64, static_cast<uint32_t>(p.pk), tt, static_cast<uint32_t>(chunks)};
  const uint64_t k_dims[4] = {64, T, static_cast<uint64_t>(p.Hkv), chunks};
  const uint64_t k_str[3] = {static_cast<uint64_t>(p.k_stride) * 2, D * 2, 128};
  const uint64_t v_str[3] = {static_cast<uint64_t>(p.v_stride) * 2, D * 2, 128};
  const uint32_t k_box[4] = {64, C::KN, 1, static_cast<uint32_t>(chunks)};
  if (!make_tensor_map_bf16(&qmap, p.q, 4, q_dims, q_str, q_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&kmap, p.k, 4, k_dims, k_str, k_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&vmap, p.v, 4, k_dims, v_str, k_box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto k = p.ctas ? packed_tc_kernel<D, true> : packed_tc_kernel<D, false>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), C::kSmem); e != cudaSuccess) return e;
  const int64_t work = static_cast<int64_t>(p.max_items) * p.heads;
  PdlLaunch l(dim3(static_cast<unsigned>(work < num_sms() ? work : num_sms())), C::kThreads, C::kSmem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, qmap, kmap, vmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool packed_tc_supported(int64_t D, int dtype) { return dtype == EXTKV_BF16 && (D == 64 || D == 128 || D == 256); }

cudaError_t launch_packed_tc(PackedParams& p, uint32_t wait_limit_plus1, cudaStream_t s, const char** name) {
  *name = "packed_tcgen05";
  p.wait_limit = wait_limit(wait_limit_plus1, kWaitPolls);
  if (p.D == 256) return launch_packed_tc_d256(p, s);
  return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace extkv
