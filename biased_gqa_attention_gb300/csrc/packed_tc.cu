// packed_tc.cu -- packed prefill on the 5th-generation tensor cores: bf16, head
// sizes 64 and 128.
//
// Bound: the tensor pipe for long prompts (4 D flops a pair against one
// exponential a pair), the softmax's instruction rate close behind it.
//
// A persistent CTA per SM takes query tiles from the plan's list (dearest
// first, rounds taken in alternating order).  An item is 256 query rows, two
// M = 128 tiles A and B of one KV head's (token, head) rows: while one tile's
// scores go through the softmax, the tensor cores work for the other.
//   warp 0       loads: Q tiles, then K and V tiles of 128 keys through a ring
//                of shared-memory units (TMA, 128-byte swizzle)
//   warps 1, 2   issue the MMAs of tile A and of tile B: PV(j-1), QK(j) for each
//                key tile; S and O live in tensor memory, P (bf16) over the
//                first half of its S.  Issuing a 128 x 128 x 16 MMA costs its
//                thread longer than the tensor pipe takes for it (64 cycles),
//                so one thread for both tiles left the pipe idle half the time
//   warps 4-7    softmax and output of tile A, a query row per thread
//   warps 8-11   the same for tile B
// (warp 3 only fills the first warpgroup, which gives its registers to the other
// two: 72 against 216 of the 168 a thread the block starts with.)
// The tensor pipe runs a thread's MMAs in order, so S_t(j) being complete
// implies that PV_t(j-1) is: a softmax warp may rescale O_t before it releases
// P_t(j) without another barrier.  O is rescaled only when a row's maximum has
// grown by more than 8 in the exponent (P then stays below 2^8, exact enough in
// bf16 and fp32 alike).
#include "internal.h"
#include "packed_tc.cuh"
#include "packed_tc.h"
#include "tma_host.h"

namespace extkv {

namespace {

using namespace packed;

constexpr int kMaxUnits = 8;

template <int D>
struct Cfg {
  static constexpr int kThreads = 384;
  static constexpr int kTile = kBM * D * 2;  // bytes of a Q, K or V tile
  static constexpr int kUnits = (232448 - 2048 - 2 * kTile) / kTile < kMaxUnits ? (232448 - 2048 - 2 * kTile) / kTile : kMaxUnits;
  static constexpr int kOffKV = 2 * kTile;
  static constexpr int kOffBar = kOffKV + kUnits * kTile;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static constexpr uint32_t kOCol = 256;  // S_A, S_B at 0 and 128; O_A, O_B from here
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, kBN, 0, 0);
  static constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, D, 0, 1);
  static_assert(kSmem <= 232448 && kUnits >= 4, "shared memory");
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t u_full[kMaxUnits], u_empty[kMaxUnits];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2];  // p_full: of each half of P
  uint64_t v_tail, drain[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// Registers of the calling warpgroup; 128 * 72 + 256 * 216 = 384 * 168.
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const PackedParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(sm + C::kOffBar);
  uint8_t* sKV = sm + C::kOffKV;
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&bar.q_full[t], 1);
      ptx::mbar_init(&bar.q_empty[t], 1);
      ptx::mbar_init(&bar.s_full[t], 1);
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
    for (int t = 0; t < 2; ++t) ptx::mbar_init(&bar.drain[t], 1);
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
  const int tt = p.tile_tok / 2;

  if (warp < 4) {
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
      ptx::mbar_arrive_expect_tx(&bar.q_full[t], C::kTile);
      ptx::tma_load_4d(sm + t * C::kTile, &qmap, &bar.q_full[t], 0, w.h0, w.row0 + w.tok0 + t * tt, 0);
      ++nq[t];
      return true;
    };
    Rounds rounds(n_work, blockIdx.x, gridDim.x);
    for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
      const Work w = work_at(p, wi);
      if (lane == 0) ok = load_q(w, 0);
      for (int kt = w.k_lo; kt < w.k_hi; ++kt) {
        const int key0 = w.row0 + kt * kBN;
        const bool tail = (kt + 1) * kBN > w.len;  // keys of the next sequence behind the last one
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
          zero_rows<D>(dst, w.len - kt * kBN, kBN, lane);
          if (lane == 0) ptx::mbar_arrive(&bar.u_full[u % C::kUnits]);
        }
        ++u;
      }
    }
    if (lane == 0 && *abort) {  // copies still in flight land before the CTA leaves
      for (int x = u >= C::kUnits ? u - C::kUnits + 1 : 0; x <= u; ++x)
        ptx::mbar_wait_bounded(&bar.u_full[x % C::kUnits], (x / C::kUnits) & 1, kWaitPolls >> 6);
      for (int t = 0; t < 2; ++t)
        if (nq[t]) ptx::mbar_wait_bounded(&bar.q_full[t], (nq[t] - 1) & 1, kWaitPolls >> 6);
      ptx::mbar_wait_bounded(&bar.v_tail, tails & 1, kWaitPolls >> 6);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ---------------- MMAs of one query tile ----------------
    if (lane == 0) {
      const int t = warp - 1;
      const uint64_t qdesc = ptx::smem_desc_sw128(ptx::smem_u32(sm + t * C::kTile), 16, 1024);
      const uint64_t kdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, 1024);
      const uint64_t vdesc = ptx::smem_desc_sw128(ptx::smem_u32(sKV), kBN * 128, 1024);
      const uint32_t ts = tbase + t * kBN, to = tbase + C::kOCol + t * D;
      int u = 0, nq = 0, np = 0;
      bool ok = true, issued = false;
      auto landed = [&](int x) { return wait_or_abort(&bar.u_full[x % C::kUnits], (x / C::kUnits) & 1, abort, lim); };
      Rounds rounds(n_work, blockIdx.x, gridDim.x);
      for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
        const Work w = work_at(p, wi);
        const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
        issued = true;
        nq += lo < hi;
        for (int kt = w.k_lo; kt <= w.k_hi; ++kt) {
          // P(kt-1) V(kt-1), then Q K(kt)^T over the S that held P(kt-1); K and V
          // are waited for first, they are mostly there
          const bool pv = kt > lo && kt <= hi, qk = kt >= lo && kt < hi;
          if (!(ok = kt == w.k_lo || landed(u - 1)) || !(ok = kt == w.k_hi || landed(u))) break;
          if (pv) {
            const bool first = kt - 1 == lo;
            if (first && nq > 1 && !(ok = wait_or_abort(&bar.o_free[t], (nq - 2) & 1, abort, lim))) break;
            const uint64_t vd = vdesc + ((((u - 1) % C::kUnits) * C::kTile) >> 4);
            for (int h = 0; h < 2 && ok; ++h) {  // the first half of the keys while the second goes through the softmax
              if (!(ok = wait_or_abort(&bar.p_full[t][h], np & 1, abort, lim))) break;
              ptx::tc_fence_after();
#pragma unroll
              for (int k = 0; k < kBN / 32; ++k) {
                const int ks = h * (kBN / 32) + k;
                ptx::umma_bf16_ts(to, ts + ks * 8, vd + ((ks * 2048) >> 4), C::kIdescPV, (!first || ks > 0) ? 1u : 0u);
              }
            }
            if (!ok) break;
            ++np;
            if (kt == hi) ptx::umma_commit(&bar.o_full[t]);
          }
          if (qk) {
            if (kt == lo && !(ok = wait_or_abort(&bar.q_full[t], (nq - 1) & 1, abort, lim))) break;
            ptx::tc_fence_after();
            const uint64_t kd = kdesc + (((u % C::kUnits) * C::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * (kBN * 128) + (k & 3) * 32) >> 4;
              ptx::umma_bf16(ts, qdesc + off, kd + off, C::kIdescQK, k > 0);
            }
            ptx::umma_commit(&bar.s_full[t]);
            if (kt == hi - 1) ptx::umma_commit(&bar.q_empty[t]);
          }
          // the slots' commits behind the products: S is what the softmax waits for
          if (kt > w.k_lo) ptx::umma_commit(&bar.u_empty[(u - 1) % C::kUnits]);
          if (kt < w.k_hi) {
            ptx::umma_commit(&bar.u_empty[u % C::kUnits]);
            u += 2;
          }
        }
      }
      // every MMA issued has completed before tensor memory is released
      if (issued) {
        ptx::umma_commit(&bar.drain[t]);
        if (!ptx::mbar_wait_bounded(&bar.drain[t], 0, kWaitPolls)) *abort = 1;
      }
    }
    __syncwarp();
  }
  } else {
    // ---------------- softmax and output ----------------
    reg_inc<216>();
    const int t = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tbase + lane_base + t * kBN, to = tbase + lane_base + C::kOCol + t * D;
    const float c = p.c;
    int ns = 0, no = 0;
    bool ok = true;
    Rounds rounds(n_work, blockIdx.x, gridDim.x);
    for (int64_t wi; ok && (wi = rounds.next()) >= 0;) {
      const Work w = work_at(p, wi);
      const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
      if (lo >= hi) continue;
      const int tok = w.tok0 + t * tt + row / p.pk;
      // the row's keys [ra, rb)
      int ra = p.window > 0 ? max(0, tok - p.window + 1) : 0, rb = p.causal ? tok + 1 : w.len;
      const bool valid = tok < w.len;
      if (!valid) ra = rb = 0;
      float m = -INFINITY, l = 0.f;
      for (int kt = lo; kt < hi; ++kt) {
        const int k0 = kt * kBN;
        if (!__all_sync(0xffffffffu, wait_or_abort(&bar.s_full[t], ns & 1, abort, lim))) {
          ok = false;
          break;
        }
        ++ns;
        ptx::tc_fence_after();
        // PV_t(kt - 1) is complete: S_t(kt) was issued after it
        softmax_tile<D>(ts, to, ra, rb, k0, c, m, l, [] { return true; },
                        [&](int h) {
                          if (lane == 0) ptx::mbar_arrive(&bar.p_full[t][h]);
                        });
      }
      if (!ok) break;
      if (!__all_sync(0xffffffffu, wait_or_abort(&bar.o_full[t], no & 1, abort, lim))) {
        ok = false;
        break;
      }
      ++no;
      ptx::tc_fence_after();
      const int64_t y0 = (static_cast<int64_t>(w.row0 + tok) * p.Hq + w.h0 + row % p.pk) * D;
      const bool in = valid && EXTKV_IN(y0, D, static_cast<int64_t>(p.T) * p.Hq * D, p.status);
      store_row<D>(to, l, in, static_cast<__nv_bfloat16*>(p.y) + y0, [&] {
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar.o_free[t]);
      });
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
  const uint32_t k_box[4] = {64, kBN, 1, static_cast<uint32_t>(chunks)};
  if (!make_tensor_map_bf16(&qmap, p.q, 4, q_dims, q_str, q_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&kmap, p.k, 4, k_dims, k_str, k_box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&vmap, p.v, 4, k_dims, v_str, k_box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto k = packed_tc_kernel<D>;
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
