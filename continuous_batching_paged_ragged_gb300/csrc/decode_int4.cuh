// The streaming warps' loop over a 4-bit cache.
//
// A block is one record (int4.cuh): K's codes, V's codes and the scales of 16 keys arrive in one bulk copy.  Blocks go in
// pairs: both blocks' scores, one softmax step, both blocks' products.
//
//   scores   S[key][head] = sum over groups g of s_K[key][g] * (sum_{d in g} c[key][d] q[d] - 8 sum_{d in g} q[d])
//   values   O[d][head]  += sum over keys of (c[key][d] - 8) * (w[key][head] * s_V[key][g(d)])
//
// with c the codes as they are stored, 1 .. 15 (8 more than what they stand for), which the tensor cores multiply in fp16.
// What bounds such a loop is instructions per block, not bytes (a record is 2.3 KB at head_dim 128 and an SM's share of
// DRAM brings one every 100 cycles), so:
//  * Unpacking: a code masked out of its word IS an fp16 number, the subnormal c * 2^-24, and its products with q or
//    with a weight are exact in the MMA's fp32 sums.  A pair of values costs a mask and a share of a shift: no conversion, no
//    exponent to set, nothing to subtract.  The factor 2^24 goes into the score's scale and into the final output.
//  * The 8: of the scores, it is the MMA's C operand, -8 sum q, summed once per task; of the values, a second MMA on
//    the same weights with a constant A (-8 * 2^-24), so that O's sums are those of the signed codes.
//  * Scores are scaled by group in fp32 (exact products of codes and q until then); a value's scale rides on its key's
//    weight, one weight fragment a group.
//  * In V's fragments every second code stays where it is in its word, 16 times as large; its output rows take that
//    back at the end.
// The weights of a block times its scales are rounded to fp16 (at most 2^-11 of each off).  So that this holds for scales
// of any size, the softmax's reference is not the running maximum but 28 - e below it (in log2 units), e the exponent field
// of the largest value scale the warp has met: weights times scales stay below 2^14 and keep 2^-24 as their smallest
// step.  l, o and the reference m belong together, whatever m is: the combiner and the merges need nothing else.
#pragma once

#include "decode.cuh"

namespace pkv {

namespace dev {
// D = A * B + C with C apart from D.
__device__ __forceinline__ void mma_16816_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                            float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one load");
  if constexpr (N == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  if constexpr (N == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ float2 halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
}  // namespace dev

// This pass's rows of a block, `nov` of them from row r0 on, quantized from the inputs exactly as the append stores them,
// over the record at `base`.  A unit is 8 values of K or V; its lane's first (units 0 .. 31) is `first`, loaded while the
// record was on its way.
template <int D>
struct NewRows {
  static constexpr int CPR = D / 8, CPT = 2 * CPR;  // units of a row; of a token (K, then V)
  static __device__ __forceinline__ uint4 load(const DecodeParams& p, int unit, int64_t token0, int g) {
    const int r = unit / CPT, kv = (unit / CPR) & 1, c = unit % CPR;
    const __half* src = (kv ? p.v_in : p.k_in) + ((size_t)(token0 + r) * p.num_kv_heads + g) * D;
    return __ldcg(reinterpret_cast<const uint4*>(src) + c);
  }
  static __device__ void store(const DecodeParams& p, uint32_t base, int r0, int nov, int64_t token0, int g, int lane, uint4 first) {
    using R = Int4Record<D>;
    for (int u0 = 0; u0 < nov * CPT; u0 += 32) {
      const int unit = u0 + lane;
      const bool in = unit < nov * CPT;
      uint4 raw = first;
      if (u0 > 0) raw = in ? load(p, unit, token0, g) : make_uint4(0, 0, 0, 0);
      const __half s = dev::int4_scale(dev::int4_group_amax(raw));  // (every lane takes part)
      if (!in) continue;
      const int r = r0 + unit / CPT, kv = (unit / CPR) & 1, c = unit % CPR;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + R::code_at(kv, r, c)), "r"(dev::int4_encode8(raw, s)) : "memory");
      if ((c & 3) == 0)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(base + R::scale_at(kv, r, c)), "h"(__half_as_ushort(s)) : "memory");
    }
    __syncwarp();
  }
};

// Row r of the record at `base` (shared memory) into slot `slot` of the cache.
template <int D>
__device__ __forceinline__ void write_row(const DecodeParams& p, uint32_t base, int r, int64_t slot, int g, int lane) {
  using R = Int4Record<D>;
  if (slot < 0 || slot >= p.num_slots) {
    if (lane == 0) dev::set_error(p.err, PKV_DEVERR_SLOT_RANGE);
    return;
  }
  unsigned char* rec = reinterpret_cast<unsigned char*>(p.cache_k) + ((size_t)(slot >> 4) * p.num_kv_heads + g) * R::BYTES;
  const int to = (int)(slot & 15);
  if (lane < 2 * R::GROUPS) {  // 16 bytes of codes a lane: K's groups, then V's
    uint32_t w[4];
    dev::lds_words<4>(base + lane * 256 + r * 16, w);
    *reinterpret_cast<uint4*>(rec + lane * 256 + to * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane < R::SCALE_ROW / 4) {
    uint32_t w[1];
    dev::lds_words<1>(base + R::SCALES + r * R::SCALE_ROW + lane * 4, w);
    *reinterpret_cast<uint32_t*>(rec + R::SCALES + to * R::SCALE_ROW + lane * 4) = w[0];
  }
}

template <int D, int G, bool W>
__device__ __forceinline__ void stream_loop_int4(const DecodeParams& p, const DecodeSmem<D, G, kKvInt4>& sm,
                                                 Streamer<D, G, kKvInt4, W>& w) {
  using T = DecodeTraits<D, G, kKvInt4>;
  using R = Int4Record<D>;
  static_assert(R::VALUES == R::GROUPS * 256, "V's codes follow K's groups");
  constexpr int NG = R::GROUPS, SW = NG / 2;  // groups of a row; 32-bit words of its K or V scales
  constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
  // -8 as the codes are scaled: 2^-24 in rows 0 .. 7 of an m-tile, 2^-20 in rows 8 .. 15
  const uint32_t minus8[4] = {0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u};
  const int lane = w.lane, warp = w.warp;
  const int qh = lane >> 2;        // this lane's score rows are keys qh and qh + 8; its q column is head qh
  const int h0 = (lane & 3) << 1;  // heads of this lane's score / output columns: h0, h0 + 1
  int shares = 0;                  // shares this warp has handed to the combiner warp
  float* my_o = sm.sh_o + warp * T::OV * T::SHL;
  float2* my_ml = sm.sh_ml + warp * kHeadsTile;
  const float scale = p.scale_log2 * 0x1p24f;
  while (w.ok && w.cur.t >= 0) {
    const TaskView d = w.cur;
    w.task_start();
    w.fill();
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // references and sums (see above)
    uint32_t top = 0;                                          // exponent field of the largest value scale met
    float shift = 28.f;                                        // 28 - top
    float o[T::MT][4];
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    const int low = W ? window_low(d.ctx, p.win.window) : 0;  // the window's first key

    if (d.nbw > 0 && w.ok) {
      uint32_t qb[T::KS][2];
      w.load_q(qb);
      // -8 sum q over each group for heads h0, h0 + 1, as the MMAs' C operand
      float c8[NG][2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = dev::halves(qb[2 * g + (i >> 1)][i & 1]);
          s += f.x + f.y;
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        c8[g][0] = __shfl_sync(0xffffffffu, s, h0 * 4) * -0x1p-21f;
        c8[g][1] = __shfl_sync(0xffffffffu, s, h0 * 4 + 4) * -0x1p-21f;
      }

      for (int j = 0; j < d.nbw && w.ok; j += 2) {
        const int n = min(2, d.nbw - j);
        uint32_t hide = 0;   // bit 2u: key qh of block u is not seen, bit 2u + 1: key qh + 8
        bool wrote = false;  // rows of this pass have gone over a record
#pragma unroll 1
        for (int u = 0; u < n; ++u) {
          const int bpos = w.block_pos(d, j + u);  // the block's first position
          const int ntok = min(kBS, d.ctx - bpos);
          // fused append: positions ov0 .. bpos + ntok - 1 of the block are this pass's tokens, whose rows come from the
          // inputs; the block holding the token's own position writes it into the cache
          const int ov0 = max(bpos, d.nst), nov = p.k_in != nullptr ? bpos + ntok - ov0 : 0;
          const int64_t token0 = d.t - (d.ctx - 1 - ov0);  // the packed token of position ov0
          const bool own = nov > 0 && d.ctx - 1 < bpos + kBS;
          uint4 first = make_uint4(0, 0, 0, 0);
          if (nov > 0 && lane < nov * NewRows<D>::CPT) first = NewRows<D>::load(p, lane, token0, d.g);
          const int64_t slot = own ? __ldcg(p.slots + d.t) : -1;
          const uint32_t base = w.wait_run(u);
          if (!w.ok) break;
          if (nov > 0) {
            NewRows<D>::store(p, base, ov0 - bpos, nov, token0, d.g, lane, first);
            if (own && slot != -1) write_row<D>(p, base, d.ctx - 1 - bpos, slot, d.g, lane);
            wrote = true;
          }
          if (ntok < kBS || (W && bpos < low)) {
            auto sees = [&](int key) { return key < ntok && (!W || bpos + key >= low || bpos + key < p.win.sinks); };
            hide |= (sees(qh) ? 0u : 1u) << (2 * u) | (sees(qh + 8) ? 0u : 2u) << (2 * u);
          }
        }
        if (!w.ok) break;
        const uint32_t base[2] = {w.run_addr(0), w.run_addr(1)};

        // ---- scores of both blocks: S^T[16 keys x 8 heads] = K Q^T ----
        float x[2][4];  // [block][key qh head h0, key qh h0 + 1, key qh + 8 h0, .. h0 + 1]
        __half2 vtop = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u][0] = x[u][1] = x[u][2] = x[u][3] = -INFINITY;
          if (u >= n) continue;
          const uint32_t row = base[u] + R::SCALES + qh * R::SCALE_ROW;
          uint32_t k0[SW], k1[SW], v0[SW], v1[SW];
          dev::lds_words<SW>(row, k0);
          dev::lds_words<SW>(row + SW * 4, v0);
          dev::lds_words<SW>(row + 8 * R::SCALE_ROW, k1);
          dev::lds_words<SW>(row + 8 * R::SCALE_ROW + SW * 4, v1);
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int gp = 0; gp < SW; ++gp) {
            uint32_t r[4];  // key qh and key qh + 8 of group 2 gp, then of group 2 gp + 1
            dev::ldsm_x4(base[u] + gp * 512 + lane * 16, r);
            const float2 f0 = dev::halves(k0[gp]), f1 = dev::halves(k1[gp]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int g = 2 * gp + h;
              const uint32_t ra = r[2 * h], rb = r[2 * h + 1];
              float c[4];
              const uint32_t a0[4] = {ra & kLo, rb & kLo, (ra >> 4) & kLo, (rb >> 4) & kLo};
              const uint32_t a1[4] = {(ra >> 8) & kLo, (rb >> 8) & kLo, (ra >> 12) & kLo, (rb >> 12) & kLo};
              dev::mma_16816_c(c, a0, qb[2 * g][0], qb[2 * g][1], c8[g][0], c8[g][1], c8[g][0], c8[g][1]);
              dev::mma_16816(c, a1, qb[2 * g + 1][0], qb[2 * g + 1][1]);
              const float fa = h ? f0.y : f0.x, fb = h ? f1.y : f1.x;
              s[0] = fmaf(c[0], fa, s[0]);
              s[1] = fmaf(c[1], fa, s[1]);
              s[2] = fmaf(c[2], fb, s[2]);
              s[3] = fmaf(c[3], fb, s[3]);
            }
          }
          const bool hid0 = hide & (1u << (2 * u)), hid1 = hide & (2u << (2 * u));
          x[u][0] = hid0 ? -INFINITY : s[0] * scale;
          x[u][1] = hid0 ? -INFINITY : s[1] * scale;
          x[u][2] = hid1 ? -INFINITY : s[2] * scale;
          x[u][3] = hid1 ? -INFINITY : s[3] * scale;
#pragma unroll
          for (int i = 0; i < SW; ++i) {  // (what lies in unseen rows may be anything)
            const uint32_t a = hid0 ? 0u : v0[i], b = hid1 ? 0u : v1[i];
            vtop = __hmax2(vtop, __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b)));
          }
        }
        // ---- one online-softmax step for the pair (log2 domain) ----
        float b0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
        float b1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
          b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, m));
          b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, m));
        }
        float r0 = m0, r1 = m1;  // the references so far, as the new shift has them
        {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(&vtop);
          const uint32_t e = __reduce_max_sync(0xffffffffu, max(v & 0xFFFFu, v >> 16)) >> 10;
          if (e > top) {
            r0 += (float)(e - top);
            r1 += (float)(e - top);
            shift -= (float)(e - top);
            top = e;
          }
        }
        const float n0 = fmaxf(r0, b0 - shift), n1 = fmaxf(r1, b1 - shift);
        const float a0 = dev::ex2_approx(m0 - n0), a1 = dev::ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u][0] = dev::ex2_approx(x[u][0] - n0);
          x[u][1] = dev::ex2_approx(x[u][1] - n1);
          x[u][2] = dev::ex2_approx(x[u][2] - n0);
          x[u][3] = dev::ex2_approx(x[u][3] - n1);
        }
        l0 = l0 * a0 + ((x[0][0] + x[0][2]) + (x[1][0] + x[1][2]));
        l1 = l1 * a1 + ((x[0][1] + x[0][3]) + (x[1][1] + x[1][3]));
        if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
          for (int mt = 0; mt < T::MT; ++mt) {
            o[mt][0] *= a0;
            o[mt][1] *= a1;
            o[mt][2] *= a0;
            o[mt][3] *= a1;
          }
        }
        // ---- O^T[d x 8 heads] += V^T P^T for both blocks ----
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (u >= n) continue;
          const uint32_t row = base[u] + R::SCALES + qh * R::SCALE_ROW + SW * 4;
          uint32_t v0[SW], v1[SW];
          dev::lds_words<SW>(row, v0);
          dev::lds_words<SW>(row + 8 * R::SCALE_ROW, v1);
          const bool hid0 = hide & (1u << (2 * u)), hid1 = hide & (2u << (2 * u));
#pragma unroll
          for (int gp = 0; gp < SW; ++gp) {
            uint32_t r[4];  // keys 2t, 2t + 1 and keys 2t + 8, 2t + 9 at dims 4 qh .. 4 qh + 3 of group 2 gp, then of 2 gp + 1
            dev::ldsm_x4_t(base[u] + R::VALUES + gp * 512 + lane * 16, r);
            const float2 f0 = dev::halves(hid0 ? 0u : v0[gp]), f1 = dev::halves(hid1 ? 0u : v1[gp]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int g = 2 * gp + h;
              const float fa = h ? f0.y : f0.x, fb = h ? f1.y : f1.x;
              const __half2 pk0 = __floats2half2_rn(x[u][0] * fa, x[u][1] * fa);
              const __half2 pk1 = __floats2half2_rn(x[u][2] * fb, x[u][3] * fb);
              const uint32_t pb0 = dev::movmatrix_t(*reinterpret_cast<const uint32_t*>(&pk0));
              const uint32_t pb1 = dev::movmatrix_t(*reinterpret_cast<const uint32_t*>(&pk1));
              const uint32_t ra = r[2 * h], rb = r[2 * h + 1];
              const uint32_t va[4] = {ra & kLo, ra & kHi, rb & kLo, rb & kHi};
              const uint32_t vb[4] = {(ra >> 8) & kLo, (ra >> 8) & kHi, (rb >> 8) & kLo, (rb >> 8) & kHi};
              dev::mma_16816(o[2 * g], va, pb0, pb1);
              dev::mma_16816(o[2 * g + 1], vb, pb0, pb1);
              dev::mma_16816(o[2 * g], minus8, pb0, pb1);
              dev::mma_16816(o[2 * g + 1], minus8, pb0, pb1);
            }
          }
        }
        if (wrote) dev::fence_proxy_async_smem();  // generic writes precede the slots' next bulk copies
        w.release_run();
        if (n > 1) w.release_run();
        w.prefetch_q();  // the next task's q, once the scheduler has published it
      }
    }
    if (!w.ok) break;

    // ---- hand this warp's share of the split to the combiner warp ----
    if (d.nbw > 0) {
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, m);
        l1 += __shfl_xor_sync(0xffffffffu, l1, m);
      }
      if (shares > 0) {  // the slot is free once the combiner warp has taken the previous share
        const bool got = cta_wait(&sm.share_empty[warp], (shares - 1) & 1, sm.abort, p.err);
        if (!__all_sync(0xffffffffu, got)) {
          w.ok = false;
          break;
        }
      }
      const int hg = lane & 3;
      if (hg < T::LG) {
        const int ci = (lane >> 2) * T::LG + hg;
#pragma unroll
        for (int r = 0; r < T::OV; ++r) my_o[r * T::SHL + ci] = o[r >> 2][r & 3] * ((r & 2) ? 0x1p20f : 0x1p24f);
        if (lane < T::LG) {
          my_ml[h0] = make_float2(m0, l0);
          my_ml[h0 + 1] = make_float2(m1, l1);
        }
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&sm.share_full[warp]);
      ++shares;
    }
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(&sm.qempty[w.k % T::QD]);  // done with the task's queue entry
    w.advance();
  }
}

}  // namespace pkv
