// paged_decode_fp8.cuh -- the tensor-core kernel of the decode over 8-bit pages;
// paged_decode_fp8.cu has the design.
#pragma once

#include "paged_decode.cuh"

namespace extkv {

namespace {

// TQ: q and y.  SP: fp16 parts that q and P are split into.
template <class C, typename TQ>
__global__ void __launch_bounds__(C::kThreads, 1)
    paged_decode_fp8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                            const PagedParams p) {
  constexpr int D = C::D, NT = C::NT, KT = C::KT, NS = C::SLOTS, KS = KT / 16, W = C::WARPS;
  constexpr int SP = sizeof(TQ) == 4 ? 2 : 1;
  constexpr int kRowsU = 8 * NT;
  constexpr int kPad = D + 4;  // rows of a partial in shared memory start in different banks
  constexpr uint32_t kFull = KT == 32 ? ~0u : (1u << (KT & 31)) - 1u;
  // A maximum that grows by less (log2 units) is let be; P stays below 2^15, and fp16
  // holds weights down to 2^-31 of the largest (fp32 q: 2^-35).
  constexpr float kGrow = SP == 2 ? 4.f : 8.f, kShift = 15.f - kGrow;
  static_assert(NS % 2 == 0 && NS >= 4, "K tiles lie in the even slots; a K tile's V tile is on its way with it");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared<C> sh;
  __shared__ LiveMasks<C> live_mask;
  __shared__ Recs<C> rec;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane >> 2, qi = lane & 3;
  init_rings<C>(kmap, vmap, sh);
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  Part<C> part;
  if (!start_part<C>(p, sh.pre, sh.warp_sum, part)) return;
  const int cta = blockIdx.x, n = part.n;
  Cursor<KT> cur = part.cur;

  bool producer = false;
  if constexpr (C::TMA) {
    producer = warp >= W;
    if (producer) produce<C>(p, kmap, vmap, smem, sh, live_mask, part);
  }
  if (!producer) {
    if (lane == 0) rec[warp] = Rec{};
    const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
    constexpr int kPieces = D / 16;  // 16-byte pieces of a row
    // place of piece ch of row r in a slot; rows of 64 bytes lie in pairs
    auto piece = [](int r, int ch) {
      if constexpr (D == 64) return static_cast<uint32_t>((r >> 1) * 128 + ((((r & 1) * 4 + ch) ^ ((r >> 1) & 7)) << 4));
      else return static_cast<uint32_t>((ch >> 3) * (KT * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
    };
    // cp.async: K, V, K, V, ... of the part's tiles; the page ids are loaded a tile
    // ahead, a tile's scales with its K and stored with its V
    Cursor<KT> ld = cur;
    TileRows<KT> rows;
    uint32_t row = ~0u, scale = 0;
    int issued = 0;
    if (!C::TMA && n > 0) rows.look_up(p, ld);
    auto issue = [&]() {
      if (C::TMA || issued >= 2 * n) return;
      const bool is_v = issued & 1;
      const int s = issued % NS;
      if (!is_v) {
        row = rows.row(p);
        const uint32_t mask = __ballot_sync(0xffffffffu, row != ~0u);
        if (lane == 0) live_mask[warp][s] = mask;
        if (row != ~0u) scale = reinterpret_cast<const uint16_t*>(p.scales)[row];
      } else if (lane < KT) {
        reinterpret_cast<uint16_t*>(sh.scales[warp][s / 2])[lane] = static_cast<uint16_t>(scale);
      }
      const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v : p.k);
#pragma unroll
      for (int i = 0; i < KT * kPieces / 32; ++i) {
        const int x = i * 32 + lane, r = x / kPieces, ch = x % kPieces;
        const uint32_t pr = __shfl_sync(0xffffffffu, row, r);
        const int64_t at = (pr != ~0u ? static_cast<int64_t>(pr) * D : 0) + ch * 16;
        cp_async_16(ring + s * C::kTile + piece(r, ch), src + at, pr != ~0u ? 16 : 0);  // no row: zeros
      }
      ++issued;
      if (is_v && issued < 2 * n) {
        ld.next(p);
        rows.look_up(p, ld);
      }
    };
    if (!C::TMA) {
      for (int s = 0; s < NS - 1; ++s) {
        issue();
        cp_async_commit();
      }
    }

    uint32_t qf[NT][SP][kPieces][2];
    uint64_t cc[NT];  // what a raw score of the thread's two columns counts, in log2 units
    float o[kPieces][NT][4];
    float m[NT][2], l[NT][2];
    uint64_t ls[NT];  // the thread's share of l
    static_assert(kRowsU * (kPad * 4 + 8) <= C::kRing, "a partial fits a warp's ring");
    int heads = 0;
    // (max in log2 units, sum) and the unnormalised rows of this warp's unit
    auto leave = [&](float2* ml, float* part, int stride) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int hr = nt * 8 + qi * 2 + h;
          if (hr < heads) {
            if (quad == 0) ml[hr] = make_float2(m[nt][h], l[nt][h]);
            float* dst = part + hr * stride + 2 * quad;
#pragma unroll
            for (int mt = 0; mt < kPieces; ++mt)
              *reinterpret_cast<float2*>(dst + mt * 16) = make_float2(o[mt][nt][h], o[mt][nt][h + 2]);
          }
        }
    };
    bool open = false;  // the unit's first tile of this warp's part has been taken
    int t_first = 0;
    int sk = 0, pk = 0;  // slot of the next tile, and its phase
    for (int it = 0; it < n; ++it) {
      if (!open) {
        open = true;
        t_first = cur.t;
        if (it == 0 && lane == 0) {
          rec[warp].n = n;
          rec[warp].b[0] = cur.b;
          rec[warp].u[0] = cur.u;
        }
        const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // the row's elements 16 kk + 4 qi .. + 3 as a k-step's B fragment: the order in
          // which a 32-bit word of K's codes gives them
          const int hr = gr * kRowsU + nt * 8 + quad;  // head within the KV head's group
          const int64_t q_at = cur.b * p.q_stride + static_cast<int64_t>(hk * p.g + hr) * D;
          const bool in = hr < p.g && q_in(p, q_at);
          const TQ* qr = static_cast<const TQ*>(p.q) + q_at + 4 * qi;
          float4 x[kPieces];
          float top = 0.f;
#pragma unroll
          for (int kk = 0; kk < kPieces; ++kk) {
            x[kk] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) {
              if constexpr (SP == 2) {
                x[kk] = *reinterpret_cast<const float4*>(qr + 16 * kk);
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(qr + 16 * kk);
                x[kk] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
              }
            }
            top = fmaxf(top, fmaxf(fmaxf(fabsf(x[kk].x), fabsf(x[kk].y)), fmaxf(fabsf(x[kk].z), fabsf(x[kk].w))));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // times a power of two that puts the largest in [2^14, 2^15): a bf16 element
          // is exact in fp16 then, or off by 2^-39 of the largest.  (Below 2^-112 times 2^126, the most that
          // leaves its inverse a normal number: the least fp32 becomes 2^-23, which fp16 holds.)
          const int e = max((__float_as_int(top) >> 23) - 127, -112);
          const float up = __int_as_float((127 + 14 - e) << 23);
          const float down = p.c * __int_as_float((127 - 14 + e) << 23);
#pragma unroll
          for (int kk = 0; kk < kPieces; ++kk) {
            const float4 s = make_float4(x[kk].x * up, x[kk].y * up, x[kk].z * up, x[kk].w * up);
            qf[nt][0][kk][0] = ptx::pack_f16x2(s.x, s.y);
            qf[nt][0][kk][1] = ptx::pack_f16x2(s.z, s.w);
            if constexpr (SP == 2) {  // the rest: off by 2^-23 of the largest at most
              const float2 a = ptx::unpack_f16x2(qf[nt][0][kk][0]), b = ptx::unpack_f16x2(qf[nt][0][kk][1]);
              qf[nt][1][kk][0] = ptx::pack_f16x2(s.x - a.x, s.y - a.y);
              qf[nt][1][kk][1] = ptx::pack_f16x2(s.z - b.x, s.w - b.y);
            }
          }
          const float d0 = __shfl_sync(0xffffffffu, down, 8 * qi), d1 = __shfl_sync(0xffffffffu, down, 8 * qi + 4);
          cc[nt] = ptx::f2(d0, d1);
          m[nt][0] = m[nt][1] = -INFINITY;
          ls[nt] = 0;
        }
#pragma unroll
        for (int mt = 0; mt < kPieces; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }
      // K has landed
      if constexpr (C::TMA) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&sh.full[warp][sk], pk, &sh.abort_flag, p.wait_limit))) break;
      } else {
        cp_async_wait<NS - 2>();
        __syncwarp();  // for every lane, and V of the tile before has been read by every lane
      }
      const uint32_t mask = live_mask[warp][sk] & key_bits<KT>(cur.keys.lo, cur.keys.hi, cur.key0());
      if (lane < KT) {  // a key's scales are taken apart once
        const uint32_t both = reinterpret_cast<const uint16_t*>(sh.scales[warp][sk / 2])[lane];
        const int kb = fp8::clamp_byte(both & 0xff), vb = fp8::clamp_byte(both >> 8);
        sh.key_scale[warp][lane] = make_float4(fp8::power(kb), static_cast<float>(vb - fp8::kBias), fp8::inverse_power(vb), 0.f);
      }
      if constexpr (!C::TMA) {
        issue();
        cp_async_commit();
      }
      const uint32_t ka = ring + sk * C::kTile;
      // a single (16 keys, 8 heads) block is summed in two chains, since an MMA waits for the
      // one before (four chains, or two of two blocks, need registers: heads of 512 take 64 us so, 61 with this)
      constexpr int CH = KS * NT >= 2 ? 1 : 2;
      float sc[KS][NT][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        float acc[CH][NT][4];
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[ch][nt][e] = 0.f;
        const int r = ks * 16 + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < kPieces; kk += 2) {
          uint32_t w[4];  // rows 0-7 and 8-15 of piece kk, then of piece kk + 1
          ptx::ldmatrix_x4(w[0], w[1], w[2], w[3], ka + piece(r, kk + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = fp8::unpack2(static_cast<uint16_t>(w[2 * x])), a1 = fp8::unpack2(static_cast<uint16_t>(w[2 * x + 1]));
            const uint32_t a2 = fp8::unpack2(static_cast<uint16_t>(w[2 * x] >> 16)), a3 = fp8::unpack2(static_cast<uint16_t>(w[2 * x + 1] >> 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int sp = 0; sp < SP; ++sp)
                ptx::mma_f16_16816(acc[(kk + x) % CH][nt], a0, a1, a2, a3, qf[nt][sp][kk + x][0], qf[nt][sp][kk + x][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[ks][nt][e] = acc[0][nt][e];
#pragma unroll
            for (int ch = 1; ch < CH; ++ch) sc[ks][nt][e] += acc[ch][nt][e];
          }
      }
      __syncwarp();  // K has been read, the keys' scales are written
      if constexpr (C::TMA) {
        if (lane == 0) ptx::mbar_arrive(&sh.empty[warp][sk]);
      }
      if (++sk == NS) {
        sk = 0;
        pk ^= 1;
      }
      // log2 of the weight of V's code: the score and the exponent of V's scale
      uint64_t ts[KS][2][NT];  // of the thread's keys ks * 16 + quad, + 8 and two columns
      uint64_t vi[KS][2];      // one over V's scale, twice
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 f = sh.key_scale[warp][ks * 16 + 8 * i + quad];
          const uint64_t kp = ptx::f2(f.x, f.x), ve = ptx::f2(f.y, f.y);
          vi[ks][i] = ptx::f2(f.z, f.z);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            ts[ks][i][nt] = ptx::fma2(ptx::f2(sc[ks][nt][2 * i], sc[ks][nt][2 * i + 1]), ptx::mul2(kp, cc[nt]), ve);
        }
      if (mask != kFull) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!((mask >> (ks * 16 + 8 * i + quad)) & 1)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) ts[ks][i][nt] = ptx::f2(-INFINITY, -INFINITY);
            }
      }
      float top[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt][0] = fmaxf(ptx::f2_lo(ts[0][0][nt]), ptx::f2_lo(ts[0][1][nt]));
        top[nt][1] = fmaxf(ptx::f2_hi(ts[0][0][nt]), ptx::f2_hi(ts[0][1][nt]));
#pragma unroll
        for (int ks = 1; ks < KS; ++ks) {
          top[nt][0] = ptx::max3(top[nt][0], ptx::f2_lo(ts[ks][0][nt]), ptx::f2_lo(ts[ks][1][nt]));
          top[nt][1] = ptx::max3(top[nt][1], ptx::f2_hi(ts[ks][0][nt]), ptx::f2_hi(ts[ks][1][nt]));
        }
        grow |= top[nt][0] > m[nt][0] + kGrow || top[nt][1] > m[nt][1] + kGrow;
      }
      // the columns' maxima, and all that counts from them, when one has grown (the first tile's: from nothing)
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = top[nt][h];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[nt][h], x);
            corr[h] = m[nt][h] == -INFINITY ? 0.f : ptx::ex2(m[nt][h] - mn);
            m[nt][h] = mn;
          }
          ls[nt] = ptx::mul2(ls[nt], ptx::f2(corr[0], corr[1]));
#pragma unroll
          for (int mt = 0; mt < kPieces; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] *= corr[e & 1];
        }
      }
      uint32_t pb[KS][NT][SP][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint64_t back = ptx::f2(m[nt][0] == -INFINITY ? 0.f : kShift - m[nt][0], m[nt][1] == -INFINITY ? 0.f : kShift - m[nt][1]);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t d = ptx::add2(ts[ks][i][nt], back);
            const float e0 = ptx::ex2(ptx::f2_lo(d)), e1 = ptx::ex2(ptx::f2_hi(d));
            ls[nt] = ptx::fma2(ptx::f2(e0, e1), vi[ks][i], ls[nt]);  // the softmax's own weights, 2^score
            // P rounded to fp16 for the product (off by at most 2^-11 of each weight, or 2^-32 of the
            // largest; two parts: 2^-22, 2^-36); the sum keeps fp32
            const uint32_t x = ptx::pack_f16x2(e0, e1);
            pb[ks][nt][0][i] = ptx::movmatrix_trans(x);
            if constexpr (SP == 2) {
              const float2 f = ptx::unpack_f16x2(x);
              pb[ks][nt][1][i] = ptx::movmatrix_trans(ptx::pack_f16x2(e0 - f.x, e1 - f.y));
            }
          }
      }
      // V has landed
      if constexpr (C::TMA) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&sh.full[warp][sk], pk, &sh.abort_flag, p.wait_limit))) break;
        if (mask != kFull) {
          // rows of masked keys, whatever they hold, become zeros: their P is 0, and 0 * NaN would be NaN
          uint8_t* vt = smem + warp * C::kRing + sk * C::kTile;
          for (int x = lane; x < KT * kPieces; x += 32) {
            const int r = x / kPieces;
            if (!((mask >> r) & 1)) *reinterpret_cast<uint4*>(vt + piece(r, x % kPieces)) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();  // before the slot's next copy
          __syncwarp();
        }
      } else {
        cp_async_wait<NS - 2>();
        __syncwarp();  // for every lane, and K of this tile has been read by every lane
        issue();
        cp_async_commit();
      }
      const uint32_t va = ring + sk * C::kTile;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int r = ks * 16 + (lane & 15);
#pragma unroll
        for (int mt = 0; mt < kPieces; mt += 2) {
          uint32_t w[4];  // keys 0-7 and 8-15 of piece mt, then of piece mt + 1; columns (2 quad, 2 quad + 1) of keys 2 qi, 2 qi + 1
          ptx::ldmatrix_x4_trans(w[0], w[1], w[2], w[3], va + piece(r, mt + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // a column's two keys side by side: output rows quad and quad + 8 are columns 2 quad and 2 quad + 1
            const uint32_t u = __byte_perm(w[2 * x], 0, 0x3120), v = __byte_perm(w[2 * x + 1], 0, 0x3120);
            const uint32_t a0 = fp8::unpack2(static_cast<uint16_t>(u)), a1 = fp8::unpack2(static_cast<uint16_t>(u >> 16));
            const uint32_t a2 = fp8::unpack2(static_cast<uint16_t>(v)), a3 = fp8::unpack2(static_cast<uint16_t>(v >> 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int sp = 0; sp < SP; ++sp)
                ptx::mma_f16_16816(o[mt + x][nt], a0, a1, a2, a3, pb[ks][nt][sp][0], pb[ks][nt][sp][1]);
          }
        }
      }
      if constexpr (C::TMA) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.empty[warp][sk]);
      }
      if (++sk == NS) {
        sk = 0;
        pk ^= 1;
      }

      const bool unit_end = cur.t == cur.tiles - 1;
      if (unit_end || it == n - 1) {
        const int hk = cur.u / p.groups, gr = cur.u - hk * p.groups;
        heads = min(kRowsU, p.g - gr * kRowsU);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            l[nt][h] = h ? ptx::f2_hi(ls[nt]) : ptx::f2_lo(ls[nt]);
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
            l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
          }
        if (unit_end && t_first == 0) {
          const int64_t y_at = (static_cast<int64_t>(cur.b) * p.Hq + hk * p.g + gr * kRowsU) * D;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float inv = l[nt][h] != 0.f ? 1.f / l[nt][h] : 0.f;
              const int hr = nt * 8 + qi * 2 + h;
              if (hr < heads && y_in(p, y_at + hr * D, D)) {
                TQ* yr = static_cast<TQ*>(p.y) + y_at + hr * D + 2 * quad;
#pragma unroll
                for (int mt = 0; mt < kPieces; ++mt) {
                  const float a = o[mt][nt][h] * inv, b = o[mt][nt][h + 2] * inv;
                  if constexpr (SP == 2) *reinterpret_cast<float2*>(yr + mt * 16) = make_float2(a, b);
                  else *reinterpret_cast<uint32_t*>(yr + mt * 16) = ptx::pack_bf16x2(a, b);
                }
              }
            }
        } else if (it < n - 1) {
          // the first unit of the part, begun before it: to the workspace, the ring is still streaming
          const int64_t at = (static_cast<int64_t>(cta) * W + warp) * kRowsU;
          if (part_in(p, at, heads, static_cast<int64_t>(p.slices) * W)) leave(p.w_ml + at, p.w_part + at * D, D);
          if (lane == 0) rec[warp].early = 1;
        } else {
          // the last unit of the part: into the ring, which has been read
          if (!C::TMA) cp_async_wait<0>();
          __syncwarp();
          float* dst = reinterpret_cast<float*>(smem + warp * C::kRing);
          leave(reinterpret_cast<float2*>(dst + kRowsU * kPad), dst, kPad);
          if (lane == 0) {
            rec[warp].late = 1;
            rec[warp].begins = t_first == 0;
            rec[warp].ends = unit_end;
            rec[warp].b[1] = cur.b;
            rec[warp].u[1] = cur.u;
          }
        }
        open = false;
      }
      cur.next(p);
    }
  }
  join_parts<C, TQ>(p, smem, sh, rec, part);
}

// Tiles of KT keys, SLOTS slots, WARPS consumers.
template <int D, int NT, int KT, int SLOTS, int WARPS, bool TMA, bool CLUSTER>
using Fp8Cfg = MmaCfg<D, NT, KT, SLOTS, WARPS, TMA, CLUSTER, false, 1, 2>;

// p.cluster: 0 where the merge kernel has to follow
template <typename TQ, class AxisC, class ClusterC>
cudaError_t launch_fp8(PagedParams& p, int variant, cudaStream_t s) {
  if (variant != kDecodeStreamK)
    p.cluster = cluster_size<ClusterC>(reinterpret_cast<const void*>(paged_decode_fp8_kernel<ClusterC, TQ>), p, variant == kDecodeCluster);
  if (variant == kDecodeCluster && !p.cluster) return cudaErrorNotSupported;
  return p.cluster ? launch_rings<ClusterC>(paged_decode_fp8_kernel<ClusterC, TQ>, p, s)
                   : launch_rings<AxisC>(paged_decode_fp8_kernel<AxisC, TQ>, p, s);
}

// Rows of codes are short, and a TMA request costs its thread the same whatever it
// carries (some 220 cycles where several lanes issue): rings are filled by requests where
// one carries 8 KB, by the consumers' own copies otherwise.  Measured (GB300, us; copies,
// requests): 32 sequences up to 6806, 16 query and 8 KV heads of 128, pages of 16: 53, 67; 131071, 65537
// and 12345, 16 and 2 heads of 128, pages of 64: 31, 34; of 64: 26, 32; 32 sequences, 16
// and 4 heads of 256, pages of 64: 55, 52, pages of 16: 55, 60; of 512: 70, 59.
template <typename TQ, int D, int NT, int KT, int SLOTS, int WARPS>
cudaError_t launch_fp8_d(PagedParams& p, int variant, cudaStream_t s) {
  constexpr bool kLong = KT * D >= 8192;
  using Copied = Fp8Cfg<D, NT, KT, SLOTS, WARPS, false, false>;
  using CopiedCluster = Fp8Cfg<D, NT, KT, SLOTS, WARPS, false, true>;
  if constexpr (kLong) {
    if (p.page_size % KT == 0 && tma_pages(p, D, 1))
      return launch_fp8<TQ, Fp8Cfg<D, NT, KT, SLOTS, WARPS, true, false>, Fp8Cfg<D, NT, KT, SLOTS, WARPS, true, true>>(p, variant, s);
  }
  return launch_fp8<TQ, Copied, CopiedCluster>(p, variant, s);
}

// Sixteen query heads a unit where the KV head has more than eight and registers allow it.
inline bool fp8_two(int64_t g, int64_t D, int dtype) { return g > 8 && D <= (dtype == EXTKV_F32 ? 128 : 256); }
// Consumer warps: as many as their registers allow (12 of 168, 8 of 255; requests need two more warps).
inline int fp8_warps(int64_t D, bool two) { return D == 64 || (D == 128 && !two) ? 12 : D == 128 ? 8 : 6; }

}  // namespace

// The tensor-core kernels for fp32 q and y (in a file of their own).
cudaError_t launch_paged_fp8_f32(const void* params, int* cluster, int variant, cudaStream_t s);

}  // namespace extkv
