// packed_tc_d256.cu -- packed prefill on the 5th-generation tensor cores for
// head size 256.
//
// Tensor memory holds S, P (bf16) and one O of 256 columns, so a CTA has one
// M = 128 query tile; QK(j + 1) is issued as soon as the softmax has S(j) in
// registers.  A K and a V tile are 64 KB each for 2048 tensor cycles: 64 bytes a
// cycle and SM from L2, about all it gives.  So two CTAs form a cluster and take
// the two query tiles of one item (the same keys): each loads half of every unit
// and multicasts it to both, which halves the reads.  What is left is shared
// memory: Q and K as operands take all of its 128 bytes a cycle during QK, V
// half of them during PV, and the tiles' writes come on top (2560 cycles for 2048
// of tensor work).
//   warp 0     loads: its Q tile; its half of each 32 KB unit of K (128 keys by
//              128 columns) and V (64 keys by 256 columns)
//   warps 1, 2 issue the MMAs, one Q K^T, the other P V: neither stands in the
//              other's waits
//   warps 3-6  softmax and output, a query row per thread
// A unit's slot is refilled when both CTAs' MMAs have read it (their commits
// arrive in both CTAs).  K has a ring of two units and V one of three: with the
// 3 and 2 the other way round, 107 us on the case below; with one ring for both,
// which each MMA warp then has to walk whole, 116 us; with units of 16 KB, 112 us.
// Measured, 7644 tokens of 16 heads in three prompts, window 1024: 105 us, 978
// TFLOP/s of the attended pairs.
#include "internal.h"
#include "packed_tc.cuh"
#include "packed_tc.h"
#include "tma_host.h"

namespace extkv {

namespace {

using namespace packed;

constexpr int D = 256;
constexpr int kThreads = 224;
constexpr int kParts = 2;  // units of a K or V tile
constexpr int kKUnits = 2, kVUnits = 3, kUnits = kKUnits + kVUnits;  // rings of K and of V, one behind the other
constexpr int kUnit = 32768;
constexpr int kVKeys = kBN / kParts;  // keys of a V unit
constexpr int kQBytes = kBM * D * 2;
constexpr int kOffKV = kQBytes;
constexpr int kOffBar = kOffKV + kUnits * kUnit;
constexpr int kSmem = kOffBar + 512 + 1024;
constexpr uint32_t kPCol = 128, kOCol = 256;  // tensor memory: S, P, O
constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, kBN, 0, 0);
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, D, 0, 1);
constexpr uint16_t kBoth = 3;
static_assert(kSmem <= 232448, "shared memory");
static_assert(kParts == 2, "a part of P per V unit, two chunks per K unit");

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t u_full[kUnits], u_empty[kUnits], v_land[kUnits];
  uint64_t s_full, s_free, p_full[2], pv_done;  // p_full: of each half of P
  uint64_t o_full, o_free, drain[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// Slot and round of the x-th unit of K or of V.
__device__ __forceinline__ int slot(bool is_v, int x) { return is_v ? kKUnits + x % kVUnits : x % kKUnits; }
__device__ __forceinline__ int round(bool is_v, int x) { return is_v ? x / kVUnits : x / kKUnits; }

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    packed_tc_d256_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const PackedParams p) {
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs: their windows start alike
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(sm + kOffBar);
  uint8_t* sKV = sm + kOffKV;
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;
  const int rank = static_cast<int>(ptx::cluster_ctarank());

  if (tid == 0) {
    ptx::mbar_init(&bar.q_full, 1);
    ptx::mbar_init(&bar.q_empty, 1);
    for (int u = 0; u < kUnits; ++u) {
      ptx::mbar_init(&bar.u_full[u], 1);
      ptx::mbar_init(&bar.u_empty[u], 2);  // an MMA warp of each CTA
      ptx::mbar_init(&bar.v_land[u], 1);
    }
    ptx::mbar_init(&bar.s_full, 1);
    ptx::mbar_init(&bar.s_free, 4);
    ptx::mbar_init(&bar.p_full[0], 4);
    ptx::mbar_init(&bar.p_full[1], 4);
    ptx::mbar_init(&bar.pv_done, 1);
    ptx::mbar_init(&bar.o_full, 1);
    ptx::mbar_init(&bar.o_free, 128);
    for (int s = 0; s < 2; ++s) ptx::mbar_init(&bar.drain[s], 1);
    bar.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tensormap(&qmap);
    ptx::prefetch_tensormap(&kmap);
    ptx::prefetch_tensormap(&vmap);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bar.tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before anything arrives on them
  ptx::tc_fence_after();
  const uint32_t tbase = bar.tmem_base;
  ptx::grid_dependency_wait();
  const int64_t n_work = static_cast<int64_t>(*p.count) * p.heads;
  Rounds rounds(n_work, blockIdx.x / 2, gridDim.x / 2);
  int armed[2] = {0, 0};  // warp 0: units whose barriers expect bytes
  uint32_t tails = 0;  // warp 0: phase of each unit's v_land

  if (warp == 0) {
    // ---------------- loads ----------------
    int nu[2] = {0, 0}, nq = 0;  // units of K and of V, items so far
    bool ok = true;
    // A K or V tile: a lane per unit waits until the unit's slot is free in both
    // CTAs, arms its barrier and sends this CTA's half to both.  (Issuing a
    // request takes a lane some 500 cycles; lanes do it side by side.)
    auto load = [&](bool is_v, const Work& w, int kt) -> bool {
      bool sent = true;
      if (lane < kParts) {
        const int x = nu[is_v] + lane, s = slot(is_v, x), r = round(is_v, x), k0 = kt * kBN + (is_v ? lane * kVKeys : 0);
        sent = r == 0 || wait_or_abort(&bar.u_empty[s], (r - 1) & 1, abort, lim);
        if (sent) {
          uint64_t* full = is_v && k0 + kVKeys > w.len ? &bar.v_land[s] : &bar.u_full[s];
          ptx::mbar_arrive_expect_tx(full, kUnit);
          ptx::tma_load_4d_multicast(sKV + s * kUnit + rank * (kUnit / 2), is_v ? &vmap : &kmap, full, 0, w.row0 + k0, w.hk,
                                     is_v ? 2 * rank : 2 * lane + rank, kBoth);
        }
      }
      ok = __all_sync(0xffffffffu, sent);
      armed[is_v] = nu[is_v] + kParts;
      if (!ok) return false;
      for (int part = 0; is_v && part < kParts; ++part) {
        const int k0 = kt * kBN + part * kVKeys, s = slot(true, nu[1] + part);
        if (k0 + kVKeys <= w.len) continue;
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.v_land[s], (tails >> s) & 1, abort, lim)))) return false;
        tails ^= 1u << s;
        zero_rows<D>(sKV + s * kUnit, max(0, w.len - k0), kVKeys, lane);
        if (lane == 0) ptx::mbar_arrive(&bar.u_full[s]);
      }
      nu[is_v] += kParts;
      return true;
    };
    for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
      const Work w = work_at<kBN, false>(p, wi);
      const bool active = rank ? w.lo[1] < w.hi[1] : w.lo[0] < w.hi[0];
      if (active) {
        if (lane == 0) {
          ok = !nq || wait_or_abort(&bar.q_empty, (nq - 1) & 1, abort, lim);
          if (ok) {
            ptx::mbar_arrive_expect_tx(&bar.q_full, kQBytes);
            ptx::tma_load_4d(sm, &qmap, &bar.q_full, 0, w.h0, w.row0 + (rank ? w.tok[1] : w.tok[0]), 0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        ++nq;
      }
      if (!load(false, w, w.k_lo)) break;
      for (int kt = w.k_lo; kt < w.k_hi && ok; ++kt) {
        if (kt + 1 < w.k_hi && !load(false, w, kt + 1)) break;
        load(true, w, kt);
      }
    }
    // (the copy of Q lands before the CTA leaves, also where another warp gives up only after this)
    if (lane == 0 && nq) ptx::mbar_wait_bounded(&bar.q_full, (nq - 1) & 1, kWaitPolls >> 6);
    __syncwarp();
  } else if (warp < 3) {
    // ---------------- MMAs: Q K^T (warp 1), P V (warp 2) ----------------
    // (K and V have rings of their own, so that each warp sees every phase of its
    // slots: a wait for one phase of a barrier passes while the phase before it is
    // still open.)
    if (lane == 0) {
      const bool pv = warp == 2;
      const uint64_t qdesc = ptx::smem_desc_sw128(ptx::smem_u32(sm), 16, 1024);
      const uint64_t kdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, 1024);
      const uint64_t vdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), kVKeys * 128, 1024);
      int u = 0, nq = 0, c = 0;  // units of its kind, items, products so far
      bool ok = true, issued = false;
      for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
        const Work w = work_at<kBN, false>(p, wi);
        const int lo = rank ? w.lo[1] : w.lo[0], hi = rank ? w.hi[1] : w.hi[0];
        issued = true;
        nq += lo < hi;
        for (int kt = w.k_lo; kt < w.k_hi && ok; ++kt) {
          const bool mine = kt >= lo && kt < hi, first = kt == lo;
          if (mine && !pv) {
            if (first && !(ok = wait_or_abort(&bar.q_full, (nq - 1) & 1, abort, lim))) break;
            // the scores before these are in the softmax's registers
            if (c > 0 && !(ok = wait_or_abort(&bar.s_free, (c - 1) & 1, abort, lim))) break;
          } else if (mine) {
            if (first && nq > 1 && !(ok = wait_or_abort(&bar.o_free, (nq - 2) & 1, abort, lim))) break;
          }
          for (int part = 0; part < kParts; ++part, ++u) {
            const int s = slot(pv, u);
            if (!(ok = wait_or_abort(&bar.u_full[s], round(pv, u) & 1, abort, lim))) break;
            if (mine && !pv) {
              ptx::tc_fence_after();
              const uint64_t kd = kdesc + ((s * kUnit) >> 4), qd = qdesc + ((part * 2 * (kBM * 128)) >> 4);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t off = ((k >> 2) * (kBN * 128) + (k & 3) * 32) >> 4;
                ptx::umma_bf16(tbase, qd + off, kd + off, kIdescQK, part > 0 || k > 0);
              }
              if (part == 1) {
                ptx::umma_commit(&bar.s_full);
                if (kt == hi - 1) ptx::umma_commit(&bar.q_empty);
              }
            } else if (mine) {
              if (!(ok = wait_or_abort(&bar.p_full[part], c & 1, abort, lim))) break;
              ptx::tc_fence_after();
              const uint64_t vd = vdesc + ((s * kUnit) >> 4);
#pragma unroll
              for (int k = 0; k < kVKeys / 16; ++k)
                ptx::umma_bf16_ts(tbase + kOCol, tbase + kPCol + (part * (kVKeys / 16) + k) * 8, vd + ((k * 2048) >> 4),
                                  kIdescPV, !first || part > 0 || k > 0);
              if (part == 1) {
                ptx::umma_commit(&bar.pv_done);
                if (kt == hi - 1) ptx::umma_commit(&bar.o_full);
              }
            }
            ptx::umma_commit_multicast(&bar.u_empty[s], kBoth);
          }
          c += mine;
        }
      }
      // every MMA issued has completed before tensor memory is released
      if (issued) {
        ptx::umma_commit(&bar.drain[warp - 1]);
        if (!ptx::mbar_wait_bounded(&bar.drain[warp - 1], 0, kWaitPolls)) *abort = 1;
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax and output ----------------
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tbase + lane_base, tp = ts + kPCol, to = ts + kOCol;
    int n = 0, no = 0;
    bool ok = true;
    for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
      const Work w = work_at<kBN, false>(p, wi);
      const int lo = rank ? w.lo[1] : w.lo[0], hi = rank ? w.hi[1] : w.hi[0];
      if (lo >= hi) continue;
      const int tok = (rank ? w.tok[1] : w.tok[0]) + row / p.pk;
      const bool valid = tok < w.len;
      int ra = p.window > 0 ? max(0, tok - p.window + 1) : 0, rb = p.causal ? tok + 1 : w.len;
      if (!valid) ra = rb = 0;
      float m = -INFINITY, l = 0.f;
      for (int kt = lo; kt < hi; ++kt, ++n) {
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.s_full, n & 1, abort, lim)))) break;
        ptx::tc_fence_after();
        Scores<kBN> s;
        s.load(ts);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.s_free);
        s.mask(ra, rb, kt * kBN);
        // PV(n - 1) is complete: P may be written, O rescaled
        bool p_free = n == 0;
        auto pv_complete = [&] {
          if (!p_free) {
            p_free = __all_sync(0xffffffffu, wait_or_abort(&bar.pv_done, (n - 1) & 1, abort, lim));
            ptx::tc_fence_after();
          }
          return p_free;
        };
        if (!(ok = take_max<D>(s.max(), to, p.c, m, l, pv_complete))) break;
        const float nm = m == -INFINITY ? 0.f : -m * p.c;
        const uint64_t c2 = ptx::f2(p.c, p.c), nm2 = ptx::f2(nm, nm);
        uint64_t ls[4] = {0, 0, 0, 0};
        uint32_t pk[32];
        s.weights<0, 64>(c2, nm2, ls, pk);
        if (!(ok = pv_complete())) break;
        ptx::tmem_st32(tp, pk);
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[0]);
        s.weights<64, 64>(c2, nm2, ls, pk);
        ptx::tmem_st32(tp + 32, pk);
        p_written();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[1]);
        const uint64_t sum = ptx::add2(ptx::add2(ls[0], ls[1]), ptx::add2(ls[2], ls[3]));
        l += ptx::f2_lo(sum) + ptx::f2_hi(sum);
      }
      if (!ok || !(ok = __all_sync(0xffffffffu, wait_or_abort(&bar.o_full, no & 1, abort, lim)))) break;
      ++no;
      ptx::tc_fence_after();
      const int64_t y0 = (static_cast<int64_t>(w.row0 + tok) * p.Hq + w.h0 + row % p.pk) * D;
      const bool in = valid && EXTKV_IN_KIND(kChkOut, y0, D, static_cast<int64_t>(p.T) * p.Hq * D, p.status);
      store_row<D>(to, l, in, static_cast<__nv_bfloat16*>(p.y) + y0, [&] {
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar.o_free);
      });
    }
  }
  ptx::grid_launch_dependents();
  ptx::tc_fence_before();
  __syncthreads();
  // Neither CTA leaves while the other's copies or commits may still reach it:
  // after the first meeting nothing more is issued, then (only after an abort)
  // what this CTA's barriers were armed for lands or was never sent.
  ptx::cluster_sync();
  if (warp == 0 && lane == 0 && *abort) {
    for (int is_v = 0; is_v < 2; ++is_v)
      for (int x = max(0, armed[is_v] - (is_v ? kVUnits : kKUnits)); x < armed[is_v]; ++x) {
        const int s = slot(is_v, x);
        ptx::mbar_wait_bounded(&bar.u_full[s], round(is_v, x) & 1, kWaitPolls >> 6);
        ptx::mbar_wait_bounded(&bar.v_land[s], (tails >> s) & 1, kWaitPolls >> 8);
      }
  }
  __syncwarp();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (tid == 0 && *abort) report(p.status, EXTKV_DEV_TIMEOUT);
  if (warp == 1) ptx::tmem_dealloc(tbase, 512);
}

}  // namespace

cudaError_t launch_packed_tc_d256(const PackedParams& p, cudaStream_t s) {
  CUtensorMap qmap, kmap, vmap;
  const uint64_t T = p.T, chunks = D / 64;
  const uint32_t tt = p.tile_tok / 2;
  const uint64_t q_dims[4] = {64, static_cast<uint64_t>(p.Hq), T, chunks};
  const uint64_t q_str[3] = {D * 2, static_cast<uint64_t>(p.q_stride) * 2, 128};
  const uint32_t q_box[4] = {64, static_cast<uint32_t>(p.pk), tt, static_cast<uint32_t>(chunks)};
  const uint64_t k_dims[4] = {64, T, static_cast<uint64_t>(p.Hkv), chunks};
  const uint64_t k_str[3] = {static_cast<uint64_t>(p.k_stride) * 2, D * 2, 128};
  const uint64_t v_str[3] = {static_cast<uint64_t>(p.v_stride) * 2, D * 2, 128};
  const uint32_t k_box[4] = {64, kBN, 1, 1}, v_box[4] = {64, kVKeys, 1, 2};
  if (!make_tensor_map_bf16(&qmap, p.q, 4, q_dims, q_str, q_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&kmap, p.k, 4, k_dims, k_str, k_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&vmap, p.v, 4, k_dims, v_str, v_box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(packed_tc_d256_kernel), kSmem); e != cudaSuccess)
    return e;
  const int64_t work = static_cast<int64_t>(p.max_items) * p.heads, clusters = num_sms() / 2;
  PdlLaunch l(dim3(static_cast<unsigned>(2 * (work < clusters ? work : clusters))), kThreads, kSmem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, packed_tc_d256_kernel, qmap, kmap, vmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace extkv
