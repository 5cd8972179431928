// packed_prefill.cu -- attention over prompts packed one after another: the
// plan kernel (the list of query tiles), the fp32 SIMT kernel and the choice
// between it and the tensor-core kernel.
#include <algorithm>

#include "internal.h"
#include "packed_plan.cuh"
#include "packed_tc.h"
#include "simt_tile.cuh"
#include "tma_host.h"

namespace extkv {

namespace {

constexpr int kSplitAt = 3;     // halves of a CTA's share of all work
constexpr int kSplitLeast = 2;  // in tiles of 128 keys

// in tiles of 128 keys
__device__ __forceinline__ int item_cost(const PackedParams& p, int len, int tok0, int tokens) {
  const int2 k = item_keys(p, len, tok0, tokens);
  return (k.y + 127) / 128 - k.x / 128;
}

// One CTA.  A causal prompt's tiles cost from one to len / 128 key tiles, so the
// list is sorted by cost, dearest first (a counting sort over kPlanThreads cost
// classes): CTAs that take items in turn then end together.  The order within a
// class follows the atomics; every item is computed alone, so no result
// depends on it.  Also checks cu_seqlens: a bad one leaves an empty list.
//
// In a small batch (p.ctas) an item that costs more than kSplitAt / 2 times a CTA's
// share of all work is listed as two of half its tokens, whose keys are split over
// the CTA's two query tiles: they take half as long one after another.  Otherwise a
// short batch waits for its longest prompt's last items.  Measured without and with:
// one prompt of 2047 rows, 8 heads of 128, 41 and 33 us; four of 50 to 3000, 8 heads
// of 64, 55 and 42; twelve of 1 to 2047, 8 heads of 128, 38.2 and 36.4; four of 900,
// 27 and 25 (splitting from one share on: 31).
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedParams p) {
  __shared__ int hist[kPlanThreads];
  __shared__ int warp_sum[kPlanThreads / 32];
  __shared__ int bad;
  __shared__ unsigned long long total_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  hist[tid] = 0;
  if (tid == 0) {
    bad = 0;
    total_s = 0;
  }
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  __syncthreads();
  bool mine_bad = false;
  for (int64_t b = tid; b <= p.B; b += kPlanThreads) {
    if (!cu_in(p, b)) break;
    const int64_t x = p.cu[b];
    mine_bad |= x < 0 || x > p.T || (b > 0 && p.cu[b - 1] > x);
  }
  if (mine_bad) bad = 1;
  __syncthreads();
  if (bad) {
    if (tid == 0) {
      report(p.status, EXTKV_DEV_BAD_SEQLENS);
      *p.count = 0;
    }
    return;
  }
  const float to_class = static_cast<float>(kPlanThreads - 1) / static_cast<float>(p.T / 128 + 2);  // an item's cost is below that
  int64_t limit = INT_MAX;  // items that cost more are split
  // Passes over all tiles: the total cost, the classes' sizes, the items.  One loop
  // (not unrolled), since the kernel's time is mostly fetching its code.
#pragma unroll 1
  for (int pass = p.ctas ? 0 : 1; pass < 3; ++pass) {
    int64_t sum = 0;
    // a warp per sequence, a lane per tile
#pragma unroll 1
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
      if (!(cu_in(p, b) && cu_in(p, b + 1))) break;
      const int row0 = static_cast<int>(p.cu[b]), len = static_cast<int>(p.cu[b + 1]) - row0;
#pragma unroll 1
      for (int64_t t = static_cast<int64_t>(lane) * p.tile_tok; t < len; t += 32 * p.tile_tok) {
        int tok = static_cast<int>(t), tokens = p.tile_tok;
        int cost = item_cost(p, len, tok, tokens);
        if (pass == 0) {
          sum += cost;
          continue;
        }
        const int split = cost > limit;
        if (split) tokens /= 2;
#pragma unroll 1
        for (int end = min(len, tok + p.tile_tok); tok < end; tok += tokens) {
          if (split) cost = (item_cost(p, len, tok, tokens) + 1) / 2;
          const int at = atomicAdd(&hist[kPlanThreads - 1 - min(kPlanThreads - 1, static_cast<int>(cost * to_class))], 1);
          if (pass == 2 && at < p.max_items && item_in(p, at))
            p.items[at] = PackedItem{row0, len, tok, split};
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0 && sum) atomicAdd(&total_s, static_cast<unsigned long long>(sum));
      __syncthreads();
      limit = max(int64_t(kSplitLeast), static_cast<int64_t>(total_s) * p.heads * kSplitAt / (2 * p.ctas));
    } else if (pass == 1) {  // each class's first place in the list
      __syncthreads();
      const int n = hist[tid];
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      int off = 0;
      for (int w = 0; w < warp; ++w) off += warp_sum[w];
      hist[tid] = off + inc - n;
      if (tid == kPlanThreads - 1) *p.count = min(off + inc, p.max_items);
      __syncthreads();
    }
  }
}

// ---- SIMT (fp32, other head sizes) ---------------------------------------------------
// A CTA takes a tile of 32 query rows (tokens by heads of one KV head), eight a
// warp, and streams the keys through two shared-memory stages that its four
// warps share.  Bound by the fp32 lanes for long prompts, by the chain of key
// tiles of one CTA for short ones: 218 rows in four prompts, 4 heads of 64, fp32:
// 20 us (23 with the rows' softmax steps one after another and q staged row by row).

constexpr int kWarps = 4;
constexpr int kTileRows = kWarps * kRows;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
__host__ __device__ constexpr int simt_stride(int D) {
  return D + 16 / static_cast<int>(sizeof(T));  // rows start in different banks
}

template <typename T, int DPL, int KT>
__global__ void __launch_bounds__(kWarps * 32, 1) packed_simt_kernel(const PackedParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = p.D;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int stride = simt_stride<T>(D), stage = 2 * KT * stride;
  T* ring = reinterpret_cast<T*>(smem);
  float* qs = reinterpret_cast<float*>(smem + 2 * stage * sizeof(T)) + warp * (kRows * D + kRows * KT);
  float* ps = qs + kRows * D;
  const int chunks = D * static_cast<int>(sizeof(T)) / 16;
  const int64_t n_work = static_cast<int64_t>(*p.count) * p.heads;
  // elements of a tensor of T rows (checked builds)
  [[maybe_unused]] auto rows_of = [&](int64_t row_stride, int heads) {
    return (p.T - 1) * row_stride + static_cast<int64_t>(heads) * D;
  };
  SimtState<DPL> st;
  for (int64_t w = blockIdx.x; w < n_work; w += gridDim.x) {
    const int64_t at = w / p.heads;
    if (!item_in(p, at)) break;
    const PackedItem item = p.items[at];
    const int h0 = static_cast<int>(w - at * p.heads) * p.pk, hk = h0 / p.g;
    const int2 keys = item_keys(p, item.len, item.tok0, p.tile_tok);
    st.clear();
    auto load = [&](int t, int s) {
      const int k0 = keys.x + t * KT;
      const uint32_t kd = ptx::smem_u32(ring + s * stage), vd = kd + KT * stride * sizeof(T);
      for (int x = tid; x < KT * chunks; x += kWarps * 32) {
        const int r = x / chunks, ch = x - r * chunks;
        bool in = k0 + r < keys.y;  // keys past the range are filled with zeros
        const int64_t row = in ? item.row0 + k0 + r : 0;
        in = in && EXTKV_IN_KIND(kChkRows, row * p.k_stride + hk * D, D, rows_of(p.k_stride, p.Hkv), p.status) &&
             EXTKV_IN_KIND(kChkRows, row * p.v_stride + hk * D, D, rows_of(p.v_stride, p.Hkv), p.status);
        const uint32_t to = r * stride * sizeof(T) + ch * 16;
        cp_async_16(kd + to, reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.k) + row * p.k_stride + hk * D) + ch * 16,
                    in ? 16 : 0);
        cp_async_16(vd + to, reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.v) + row * p.v_stride + hk * D) + ch * 16,
                    in ? 16 : 0);
      }
    };
    const int nt = (keys.y - keys.x + KT - 1) / KT;
    load(0, 0);
    cp_async_commit();
    simt_stage_q<T, DPL>(qs, D, p.c, [&](int r) -> const T* {
      const int row = warp * kRows + r, tok = item.tok0 + row / p.pk;
      const int64_t q_at = (item.row0 + tok) * p.q_stride + static_cast<int64_t>(h0 + row % p.pk) * D;
      return tok < item.len && EXTKV_IN_KIND(kChkRows, q_at, D, rows_of(p.q_stride, p.Hq), p.status)
                 ? static_cast<const T*>(p.q) + q_at
                 : nullptr;
    });
    for (int t = 0; t < nt; ++t) {
      if (t + 1 < nt) load(t + 1, (t + 1) & 1);
      cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      const int k0 = keys.x + t * KT;
      int lo[kRows], hi[kRows];
      bool any = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int tok = item.tok0 + (warp * kRows + r) / p.pk;
        int a = p.window > 0 ? max(0, tok - p.window + 1) : 0, b = p.causal ? tok + 1 : item.len;
        if (tok >= item.len) a = b = 0;
        lo[r] = min(max(a - k0, 0), KT);
        hi[r] = min(max(b - k0, 0), KT);
        any |= lo[r] < hi[r];
      }
      const T* kt = ring + (t & 1) * stage;
      if (any) simt_tile<T, DPL, KT>(st, kt, kt + KT * stride, stride, qs, ps, D, lo, hi);
      __syncthreads();
    }
    st.reduce();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = warp * kRows + r, tok = item.tok0 + row / p.pk;
      if (tok < item.len) {
        const float inv = st.l[r] != 0.f ? 1.f / st.l[r] : 0.f;
        const int64_t y0 = (static_cast<int64_t>(item.row0 + tok) * p.Hq + h0 + row % p.pk) * D;
        T* y = static_cast<T*>(p.y);
        if (EXTKV_IN_KIND(kChkOut, y0, D, static_cast<int64_t>(p.T) * p.Hq * D, p.status)) {
#pragma unroll
          for (int i = 0; i < DPL; ++i) {
            const int d = lane + 32 * i;
            if (d < D) y[y0 + d] = Elem<T>::from_float(st.acc[r][i] * inv);
          }
        }
      }
    }
    __syncthreads();
  }
}

template <typename T, int DPL, int KT>
cudaError_t launch_simt(const PackedParams& p, cudaStream_t s) {
  const size_t smem = 2 * 2 * KT * simt_stride<T>(p.D) * sizeof(T) +
                      static_cast<size_t>(kWarps) * (kRows * p.D + kRows * KT) * 4;
  auto k = packed_simt_kernel<T, DPL, KT>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), smem); e != cudaSuccess) return e;
  const int64_t blocks = std::min<int64_t>(static_cast<int64_t>(p.max_items) * p.heads, int64_t(num_sms()) * 2);
  PdlLaunch l(dim3(static_cast<unsigned>(blocks)), kWarps * 32, smem, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_d(const PackedParams& p, cudaStream_t s) {
  if (p.D <= 64) return launch_simt<T, 2, 32>(p, s);
  if (p.D <= 128) return launch_simt<T, 4, 32>(p, s);
  if (p.D <= 256) return launch_simt<T, 8, 16>(p, s);
  return launch_simt<T, 16, 8>(p, s);
}

// The largest power of two that divides g, at most `cap`.
int pack_heads(int64_t g, int cap) {
  int pk = 1;
  while (pk < cap && g % (2 * pk) == 0) pk *= 2;
  return pk;
}

// Rows of a work item and the query heads packed into it.  The tensor-core
// kernel's query tiles are M = 128 rows.
struct Shape {
  bool tc, split;  // split: items may be of half the rows
  int rows, pk;
};

Shape shape_of(int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  Shape s;
  s.tc = packed_tc_supported(D, dtype);
  s.split = s.tc && D != 256;
  s.rows = s.tc ? kPackedTcRows : kTileRows;
  s.pk = pack_heads(Hq / Hkv, s.tc ? 128 : kTileRows);
  return s;
}

int64_t max_items(const Shape& s, int64_t T, int64_t B) {
  return T / (s.rows / s.pk / (s.split ? 2 : 1)) + B + 1;
}

}  // namespace

size_t packed_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  return 256 + ((max_items(shape_of(Hq, Hkv, D, dtype), T, B) * sizeof(PackedItem) + 255) & ~size_t(255));
}

cudaError_t launch_packed(const PackedArgs& a, const char** name) {
  PackedParams p{};
  p.y = a.y;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.cu = a.cu_seqlens;
  p.c = a.scale * kLog2e;
  p.causal = a.causal != 0;
  p.window = a.window > 0 ? a.window : 0;
  p.T = static_cast<int>(a.T);
  p.B = static_cast<int>(a.B);
  p.Hq = static_cast<int>(a.Hq);
  p.Hkv = static_cast<int>(a.Hkv);
  p.g = p.Hq / p.Hkv;
  p.D = static_cast<int>(a.D);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  const Shape sh = shape_of(a.Hq, a.Hkv, a.D, a.dtype);
  p.pk = sh.pk;
  p.tile_tok = sh.rows / sh.pk;
  p.heads = p.Hq / p.pk;
  p.max_items = static_cast<int>(max_items(sh, a.T, a.B));
  // Three tiles and more for two CTAs balance without splits, whose pass over the list
  // then costs more than it gives (2047 rows of 32 heads, 256 tiles: 44 us without,
  // 47 with); 256 rows and fewer have no item to split.
  p.ctas = sh.split && 2 * (a.T / p.tile_tok) * p.heads < 3 * num_sms() && a.T > 128 * kSplitLeast ? num_sms() : 0;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.count = reinterpret_cast<int*>(ws);
  p.items = reinterpret_cast<PackedItem*>(ws + 256);
  p.status = a.status;
  PdlLaunch l(dim3(1), kPlanThreads, 0, a.stream);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, packed_plan_kernel, p);
  if (e != cudaSuccess) return e;
  *name = a.dtype == EXTKV_F32 ? "packed_simt_f32" : "packed_simt_bf16";
  e = sh.tc                    ? launch_packed_tc(p, a.wait_limit_plus1, a.stream, name)
      : a.dtype == EXTKV_F32 ? launch_simt_d<float>(p, a.stream) : launch_simt_d<__nv_bfloat16>(p, a.stream);
  if (e == cudaSuccess) note_launches(2);
  return e;
}

}  // namespace extkv
