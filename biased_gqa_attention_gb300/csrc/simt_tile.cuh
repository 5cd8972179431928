// simt_tile.cuh -- a warp's online-softmax step over one tile of keys in
// shared memory, in fp32 on the SIMT lanes: the exact path of the paged decode
// and the packed prefill for fp32 and for head sizes without a tensor-core
// kernel.
//
// A warp holds kRows query rows that share a KV head.  Scores: lane = (key,
// part), the 32 / KT parts of a key taking every (32/KT)-th 16-byte vector of
// its row; a vector of K is multiplied with the same vector of all rows, so one
// shared load feeds kRows * VW multiply-adds.  Output: lane owns columns
// lane + 32 i, and a value of V feeds kRows multiply-adds.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace extkv {

constexpr int kRows = 8;

template <typename T>
struct SimtVec {
  static constexpr int N = 16 / sizeof(T);
};

// 16 bytes of shared memory as fp32
__device__ __forceinline__ void load_vec(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x;
  f[1] = v.y;
  f[2] = v.z;
  f[3] = v.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// DPL: columns per lane (head size rounded up, over 32); KT: keys per tile.
// l is this lane's share of the row's sum: reduce() adds the lanes up.
template <int DPL>
struct SimtState {
  float m[kRows], l[kRows];
  float acc[kRows][DPL];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < DPL; ++i) acc[r][i] = 0.f;
    }
  }
  __device__ __forceinline__ void reduce() {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int r = 0; r < kRows; ++r) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
  }
};

// kRows rows of q (row r at at(r), or nowhere: nullptr) into shared memory as fp32
// times `scale`: 16 bytes a lane, all loads of a lane in flight together.
template <typename T, int DPL, class F>
__device__ __forceinline__ void simt_stage_q(float* qs, int D, float scale, F at) {
  constexpr int VW = SimtVec<T>::N, kLoads = kRows * DPL / VW;  // 16-byte pieces of a lane, D = 32 DPL
  const int lane = threadIdx.x & 31, per_row = D / VW;
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int x = lane + 32 * i, r = x / per_row;
    const T* row = r < kRows ? at(r) : nullptr;
    v[i] = row ? *reinterpret_cast<const uint4*>(row + (x - r * per_row) * VW) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int x = lane + 32 * i;
    if (x < kRows * per_row) {
      float f[VW];
      load_vec(reinterpret_cast<const T*>(&v[i]), f);
#pragma unroll
      for (int e = 0; e < VW; ++e) qs[x * VW + e] = f[e] * scale;
    }
  }
}

// One tile.  ks, vs: rows of `stride` elements (a multiple of 16 bytes), KT of
// each; qs: [kRows][D] fp32, already scaled (rows that do not exist: zeros); ps:
// [KT][kRows] scratch of this warp; lo[r], hi[r]: the row's allowed keys in the
// tile, [lo, hi) of [0, KT).  Masked keys are left out by selection, and the V
// rows of keys that no row attends are not touched.  Every step runs over all
// rows at once, so that their shuffles and exponentials overlap.
template <typename T, int DPL, int KT>
__device__ __forceinline__ void simt_tile(SimtState<DPL>& st, const T* ks, const T* vs, int stride, const float* qs,
                                          float* ps, int D, const int (&lo)[kRows], const int (&hi)[kRows]) {
  constexpr int VW = SimtVec<T>::N;
  constexpr int LPK = 32 / KT;
  const int lane = threadIdx.x & 31;
  const int key = lane / LPK, part = lane % LPK;
  float s[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) s[r] = 0.f;
  const T* krow = ks + key * stride;
#pragma unroll 4
  for (int c = part * VW; c < D; c += LPK * VW) {
    float kf[VW];
    load_vec(krow + c, kf);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int e = 0; e < VW; e += 4) {
        const float4 qv = *reinterpret_cast<const float4*>(qs + r * D + c + e);
        s[r] = fmaf(qv.x, kf[e], s[r]);
        s[r] = fmaf(qv.y, kf[e + 1], s[r]);
        s[r] = fmaf(qv.z, kf[e + 2], s[r]);
        s[r] = fmaf(qv.w, kf[e + 3], s[r]);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < LPK; o <<= 1)
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
  float top[kRows];
  int any_lo = KT, any_hi = 0;  // keys some row attends
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (!(key >= lo[r] && key < hi[r])) s[r] = -INFINITY;
    top[r] = s[r];
    any_lo = min(any_lo, lo[r] < hi[r] ? lo[r] : KT);
    any_hi = max(any_hi, lo[r] < hi[r] ? hi[r] : 0);
  }
#pragma unroll
  for (int o = 16; o >= LPK; o >>= 1)
#pragma unroll
    for (int r = 0; r < kRows; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
  float pr[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float m_new = fmaxf(st.m[r], top[r]);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float corr = st.m[r] == -INFINITY ? 0.f : exp2f(st.m[r] - ref);
    const bool live = key >= lo[r] && key < hi[r];
    pr[r] = live ? exp2f(s[r] - ref) : 0.f;
    st.l[r] = fmaf(st.l[r], corr, part == 0 ? pr[r] : 0.f);
    st.m[r] = m_new;
#pragma unroll
    for (int i = 0; i < DPL; ++i) st.acc[r][i] *= corr;
  }
  if (part == 0) {
#pragma unroll
    for (int r = 0; r < kRows; r += 4)
      *reinterpret_cast<float4*>(ps + key * kRows + r) = make_float4(pr[r], pr[r + 1], pr[r + 2], pr[r + 3]);
  }
  __syncwarp();
#pragma unroll 4
  for (int j = any_lo; j < any_hi; ++j) {
    float pj[kRows];
#pragma unroll
    for (int r = 0; r < kRows; r += 4) {
      const float4 v = *reinterpret_cast<const float4*>(ps + j * kRows + r);
      pj[r] = v.x;
      pj[r + 1] = v.y;
      pj[r + 2] = v.z;
      pj[r + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < DPL; ++i) {
      const int d = lane + 32 * i;
      const float v = d < D ? Elem<T>::to_float(vs[j * stride + d]) : 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) st.acc[r][i] = fmaf(pj[r], v, st.acc[r][i]);
    }
  }
  __syncwarp();
}

}  // namespace extkv
