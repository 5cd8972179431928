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
};

// One tile.  ks, vs: rows of `stride` elements (a multiple of 16 bytes), KT of
// each, finite or to be masked; qs: [kRows][D] fp32, already scaled; ps: [kRows][KT]
// scratch of this warp; lo[r], hi[r]: the row's allowed keys in the tile,
// [lo, hi) of [0, KT).  Masked keys are left out by selection and their V rows
// are not touched by a row that does not attend them, unless another row does.
template <typename T, int DPL, int KT>
__device__ __forceinline__ void simt_tile(SimtState<DPL>& st, const T* ks, const T* vs, int stride, const float* qs,
                                          float* ps, int D, const int (&lo)[kRows], const int (&hi)[kRows], int n_rows) {
  constexpr int VW = SimtVec<T>::N;
  constexpr int LPK = 32 / KT;
  const int lane = threadIdx.x & 31;
  const int key = lane / LPK, part = lane % LPK;
  float s[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) s[r] = 0.f;
  const T* krow = ks + key * stride;
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
  int any_lo = KT, any_hi = 0;  // keys some row attends
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r >= n_rows) break;
#pragma unroll
    for (int o = 1; o < LPK; o <<= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
    const bool live = key >= lo[r] && key < hi[r];
    const float x = live ? s[r] : -INFINITY;
    float mt = x;
#pragma unroll
    for (int o = 16; o >= LPK; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const float m_new = fmaxf(st.m[r], mt);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float corr = st.m[r] == -INFINITY ? 0.f : exp2f(st.m[r] - ref);
    const float pr = live ? exp2f(x - ref) : 0.f;
    float sum = pr;
#pragma unroll
    for (int o = 16; o >= LPK; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    st.l[r] = fmaf(st.l[r], corr, sum);
    st.m[r] = m_new;
    if (part == 0) ps[r * KT + key] = pr;
    if (corr != 1.f) {
#pragma unroll
      for (int i = 0; i < DPL; ++i) st.acc[r][i] *= corr;
    }
    any_lo = min(any_lo, lo[r]);
    any_hi = max(any_hi, hi[r]);
  }
  __syncwarp();
  for (int j = any_lo; j < any_hi; ++j) {
    float pj[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) pj[r] = r < n_rows ? ps[r * KT + j] : 0.f;
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
