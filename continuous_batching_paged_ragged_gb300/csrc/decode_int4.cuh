// Decode over a 4-bit cache: the streaming warps' loop, and the kernel around it.
//
// A block is one record (int4.cuh): K's codes, V's codes and the scales of 16 keys arrive together.  Blocks go in
// pairs: both blocks' scores, one softmax step, both blocks' products, in one straight line of code whose chains overlap.
//
//   scores   S[key][head] = sum over groups g of s_K[key][g] * sum_{d in g} code[key][d] q[d]
//   values   O[d][head]  += sum over keys of (code[key][d] s_V[key][g(d)]) * w[key][head]
//
// What bounds such a loop is instructions per block as much as bytes (a record is 2.3 KB at head_dim 128, an SM's share of
// DRAM brings one every 100 cycles, and a quarter of the SM works on one for 390: 220 at head_dim 64 for 50, 810 at 256 for
// 200), so the work on a code is what it can be in packed fp16: a mask under an exponent makes
// 1024 + c or 1024 + 16 c of it (c = code + 8, as it is stored), one fused multiply-add the code itself.  Scores are
// scaled by group in fp32, on the exact sums of 32 products.  Values are multiplied by their scales in fp16, which is exact
// (a code times its scale is an fp16 number, subnormal or not).
// The softmax's reference moves only when a weight would pass 2^15, and then to 2^-4 of the largest: most pairs need neither
// a reduction over the warp nor a rescaling of O.  (Weights are rounded to fp16 for the product, at most 2^-11 of each off;
// l, o and the reference m belong together, whatever m is: the combiner and the merges need nothing else.)
// Tried: codes as fp16 subnormals c * 2^-24, straight out of the mask, and the 8 taken away by MMAs of its own: a fifth fewer
// instructions, but the tensor core lines such products up by their exponents and cuts off what is 2^-14 of a key's scale.
// And the keys' upper codes as 64 + c, straight out of the mask, the 72 q too much taken away in the products' first
// accumulator: 365 in place of 390 cycles a block, nothing of a pass (the offsets' registers cost a tenth at head_dim 256).
#pragma once

#include "decode.cuh"

namespace pkv {

namespace dev {
// D = A * B.
__device__ __forceinline__ void mma_16816_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
}  // namespace dev

// This pass's rows of a block, `nov` of them from row r0 on, quantized from the inputs exactly as the append stores them,
// over the record at `base`.  A unit is 8 values of K or V, a lane's at a time.
template <int D>
struct NewRows {
  static constexpr int CPR = D / 8, CPT = 2 * CPR;  // units of a row; of a token (K, then V)
  static __device__ __forceinline__ uint4 load(const DecodeParams& p, int unit, int64_t token0, int g) {
    const int r = unit / CPT, kv = (unit / CPR) & 1, c = unit % CPR;
    const __half* src = (kv ? p.v_in : p.k_in) + ((size_t)(token0 + r) * p.num_kv_heads + g) * D;
    return __ldcg(reinterpret_cast<const uint4*>(src) + c);
  }
  static __device__ void store(const DecodeParams& p, uint32_t base, int r0, int nov, int64_t token0, int g, int lane) {
    using R = Int4Record<D>;
    for (int unit = lane; unit - lane < nov * CPT; unit += 32) {
      const bool in = unit < nov * CPT;
      const uint4 raw = in ? load(p, unit, token0, g) : make_uint4(0, 0, 0, 0);
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

// The pair of codes in bits 0 .. 3 (lo) or 4 .. 7 (hi) of a word's halves.
namespace dev {
// (x & mask) | bits, in one instruction (from the expression the compiler makes two: 490 in place of 390 cycles a block and
// scheduler at head_dim 128).
__device__ __forceinline__ uint32_t masked_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ __half2 codes_lo(uint32_t x) {  // 1024 + c - 1032
  return __hadd2(as_half2(masked_or(x, 0x000F000Fu, 0x64006400u)), as_half2(0xE408E408u));
}
__device__ __forceinline__ __half2 codes_hi(uint32_t x) {  // (1024 + 16 c) / 16 - 72
  return __hfma2(as_half2(masked_or(x, 0x00F000F0u, 0x64006400u)), as_half2(0x2C002C00u), as_half2(0xD480D480u));
}
}  // namespace dev

// One step over a pair of blocks, whose records are at base[0] and base[1] in shared memory: scores, the softmax's step, values.
// hide: bit 2u, this lane's key qh of block u is not seen, bit 2u + 1: key qh + 8.  References m, sums l, outputs o.
template <int D>
__device__ __forceinline__ void attend_pair(const uint32_t (&base)[2], uint32_t hide, const uint32_t (&qb)[D / 16][2], float scale,
                                            int lane, float& m0, float& m1, float& l0, float& l1, float (&o)[D / 16][4]) {
  using R = Int4Record<D>;
  static_assert(R::VALUES == R::GROUPS * 256, "V's codes follow K's groups");
  constexpr int NG = R::GROUPS, SW = NG / 2;  // groups of a row; 32-bit words of its K or V scales
  constexpr int LW = SW < 2 ? SW : 2;         // of which so many are loaded at once (more cost registers)
  constexpr float kCap = 15.f, kTop = 4.f;    // log2 of the largest weight allowed, and of the largest after a move
  const int qh = lane >> 2;        // this lane's score rows are keys qh and qh + 8; its q column is head qh
  const int h0 = (lane & 3) << 1;  // heads of this lane's score / output columns: h0, h0 + 1; its value columns are keys h0, h0 + 1
  // ---- scores of both blocks: S^T[16 keys x 8 heads] = K Q^T ----
  float s[2][4];  // [block][key qh head h0, key qh h0 + 1, key qh + 8 h0, .. h0 + 1]
  {
    uint32_t k0[2][LW], k1[2][LW];
#pragma unroll
    for (int u = 0; u < 2; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
    for (int gp = 0; gp < SW; ++gp) {
      if (gp % LW == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          dev::lds_words<LW>(base[u] + R::SCALES + qh * R::SCALE_ROW + gp * 4, k0[u]);
          dev::lds_words<LW>(base[u] + R::SCALES + (qh + 8) * R::SCALE_ROW + gp * 4, k1[u]);
        }
      }
      uint32_t r[2][4];  // key qh and key qh + 8 of group 2 gp, then of group 2 gp + 1
      float c[2][2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) dev::ldsm_x4(base[u] + gp * 512 + lane * 16, r[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t ra = r[u][2 * h], rb = r[u][2 * h + 1];
          const uint32_t a[4] = {dev::as_word(dev::codes_lo(ra)), dev::as_word(dev::codes_lo(rb)),
                                 dev::as_word(dev::codes_hi(ra)), dev::as_word(dev::codes_hi(rb))};
          dev::mma_16816_0(c[u][h], a, qb[4 * gp + 2 * h][0], qb[4 * gp + 2 * h][1]);
        }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t ra = r[u][2 * h] >> 8, rb = r[u][2 * h + 1] >> 8;
          const uint32_t a[4] = {dev::as_word(dev::codes_lo(ra)), dev::as_word(dev::codes_lo(rb)),
                                 dev::as_word(dev::codes_hi(ra)), dev::as_word(dev::codes_hi(rb))};
          dev::mma_16816(c[u][h], a, qb[4 * gp + 2 * h + 1][0], qb[4 * gp + 2 * h + 1][1]);
        }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 f0 = dev::halves(k0[u][gp % LW]), f1 = dev::halves(k1[u][gp % LW]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float fa = h ? f0.y : f0.x, fb = h ? f1.y : f1.x;
          s[u][0] = fmaf(c[u][h][0], fa, s[u][0]);
          s[u][1] = fmaf(c[u][h][1], fa, s[u][1]);
          s[u][2] = fmaf(c[u][h][2], fb, s[u][2]);
          s[u][3] = fmaf(c[u][h][3], fb, s[u][3]);
        }
      }
    }
  }
  if (hide != 0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (hide & (1u << (2 * u))) s[u][0] = s[u][1] = -INFINITY;
      if (hide & (2u << (2 * u))) s[u][2] = s[u][3] = -INFINITY;
    }
  }
  // ---- one online-softmax step for the pair (log2 domain): the references move if some weight would pass its cap.  Scores are
  // rounded before the references are taken and subtracted, so that the largest weight is what the reference makes it at
  // any size (in one fused operation with the subtraction, scores of 2^28 had weights off by 2^16) ----
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[u][i] = __fmul_rn(s[u][i], scale);  // (not to be fused)
  float b0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
  float b1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
  if (__any_sync(0xffffffffu, b0 - m0 > kCap || b1 - m1 > kCap)) {
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) {
      b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, m));
      b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, m));
    }
    const float n0 = b0 - m0 > kCap ? b0 - kTop : m0, n1 = b1 - m1 > kCap ? b1 - kTop : m1;
    const float a0 = dev::ex2_approx(m0 - n0), a1 = dev::ex2_approx(m1 - n1);
    m0 = n0;
    m1 = n1;
    l0 *= a0;
    l1 *= a1;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      o[mt][0] *= a0;
      o[mt][1] *= a1;
      o[mt][2] *= a0;
      o[mt][3] *= a1;
    }
  }
  uint32_t pb[2][2];  // P^T as the MMAs' B operand: k = keys, n = heads
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float p0 = dev::ex2_approx(s[u][0] - m0), p1 = dev::ex2_approx(s[u][1] - m1);
    const float p2 = dev::ex2_approx(s[u][2] - m0), p3 = dev::ex2_approx(s[u][3] - m1);
    l0 += p0 + p2;
    l1 += p1 + p3;
    pb[u][0] = dev::movmatrix_t(dev::as_word(__floats2half2_rn(p0, p1)));
    pb[u][1] = dev::movmatrix_t(dev::as_word(__floats2half2_rn(p2, p3)));
  }
  // ---- O^T[d x 8 heads] += V^T P^T for both blocks ----
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t v0[2][LW], v1[2][LW];  // value scales: [keys h0, h0 + 1][groups], the same for keys h0 + 8, h0 + 9
#pragma unroll
    for (int gp = 0; gp < SW; ++gp) {
      if (gp % LW == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dev::lds_words<LW>(base[u] + R::SCALES + (h0 + i) * R::SCALE_ROW + (SW + gp) * 4, v0[i]);
          dev::lds_words<LW>(base[u] + R::SCALES + (h0 + 8 + i) * R::SCALE_ROW + (SW + gp) * 4, v1[i]);
        }
      }
      uint32_t r[4];  // keys h0, h0 + 1 and keys h0 + 8, h0 + 9 at dims 4 qh .. 4 qh + 3 of group 2 gp, then of 2 gp + 1
      dev::ldsm_x4_t(base[u] + R::VALUES + gp * 512 + lane * 16, r);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __half2 sa = dev::as_half2(__byte_perm(v0[0][gp % LW], v0[1][gp % LW], h ? 0x7632 : 0x5410));
        const __half2 sb = dev::as_half2(__byte_perm(v1[0][gp % LW], v1[1][gp % LW], h ? 0x7632 : 0x5410));
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // dims 4 qh + 2 e (rows 0 .. 7 of the tile) and 4 qh + 2 e + 1
          const uint32_t ra = r[2 * h] >> (8 * e), rb = r[2 * h + 1] >> (8 * e);
          const uint32_t a[4] = {dev::as_word(__hmul2(dev::codes_lo(ra), sa)), dev::as_word(__hmul2(dev::codes_hi(ra), sa)),
                                 dev::as_word(__hmul2(dev::codes_lo(rb), sb)), dev::as_word(__hmul2(dev::codes_hi(rb), sb))};
          dev::mma_16816(o[4 * gp + 2 * h + e], a, pb[u][0], pb[u][1]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------------
// The 4-bit cache's decode kernel: one CTA per SM, the tasks and the scheduler warp of the other formats, a combiner warp, and
// producer warps that copy a task's records, two blocks a stage, for the streaming warps.  A pair of blocks is 4.6 KB at
// head_dim 128, and an SM's share of DRAM brings one every 200 cycles: with the copies issued by the streaming warps themselves
// (as the larger blocks' are) a pair cost 700 cycles of issuing and waiting beside 1,200 of arithmetic, with 16-byte copies by
// all lanes more; in stages that all streaming warps share, a wait may meet its stage's phase two rounds off.
// Measured: one row of 700 tokens, 12 / 2 heads at d 128, 7.4 us; 256 rows of up to 8192 tokens 75.7 us, 3.9 TB/s; four rows of
// 262144 tokens, 16 / 4 heads at d 256, 236 us, 5.1 TB/s; 200 rows behind a window of 2048, 8 / 2 heads at d 64, 22 us; with the
// append fused 7.9, 75.7, 236 and 23.  Of the
// 76 us the warps compute for 44; the launch and its first loads take 4, what a task costs its warps besides its pairs 15 (its
// q, its share, waits between tasks), the combiner's last tasks and merges 7 and SMs that end early the rest.
// ---------------------------------------------------------------------------------------------------

// Waits for every lane's own barrier (lanes without `mine` have none): all are tested at once, and the wait proper is the whole
// warp's on the first that is not there.  (With each lane in a wait of its own they suspend the warp one after another, long
// after the last barrier has completed: one row of 700 tokens took 10.3 in place of 7.9 us.)  Behind it every lane sees what
// lies behind every lane's barrier.  False: a wait ran out.
__device__ __forceinline__ bool cta_wait_lanes(uint64_t* bar, uint32_t parity, bool mine, volatile int* abort, int32_t* err) {
  const uint32_t mine_at = dev::smem_addr(bar);
  for (;;) {
    const uint32_t left = __ballot_sync(0xffffffffu, mine && !dev::mbar_test_wait(bar, parity));
    if (left == 0) {
      __syncwarp();  // (a lane's test orders that lane's reads alone, and a ballot orders none)
      return true;
    }
    const int l = __ffs(left) - 1;
    const uint32_t at = __shfl_sync(0xffffffffu, mine_at, l), ph = __shfl_sync(0xffffffffu, parity, l);
    const bool got = cta_wait(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(at)), ph, abort, err);
    if (!__all_sync(0xffffffffu, got)) return false;
  }
}

// A task as the streaming warps see it.
template <int D, int G, bool W>
struct Int4Task {
  using T = DecodeTraits<D, G, kKvInt4>;
  int t, g, ctx, nst, base, nb;
  typename T::Jump jump;
  __device__ Int4Task(const DecodeParams& p, const typename T::Task& e) {
    const int4 rec = e.rec;
    t = rec.x;
    g = rec.y & 0xFF;
    ctx = rec.w;
    base = (rec.y >> 8) * split_size<W>(p, ctx);
    nst = e.nst;
    nb = e.nb;
    jump = W ? e.jump : 0;
  }
  __device__ __forceinline__ int pairs() const { return (nb + 1) / 2; }
  // First position of the split's block b.
  __device__ __forceinline__ int block_pos(int b) const {
    const int gap = W && b >= (int)(jump & ((1u << T::JB) - 1)) ? (int)(jump >> T::JB) : 0;
    return (base + b + gap) * kBS;
  }
  // Whether block b is not simply sixteen cached keys that the token sees: it has keys past the context, rows of this pass
  // (append fused), or keys between the sinks and the window, whose first key is `low`.
  __device__ __forceinline__ bool edge(const DecodeParams& p, int b, int low) const {
    const int bpos = block_pos(b);
    return bpos + kBS > ctx || (p.k_in != nullptr && bpos + kBS > nst) || (W && bpos < low && bpos + kBS > p.win.sinks);
  }
};

// Such a block, whose record is at `base`.  Fused append: the rows of this pass's tokens in it come from the inputs, and the
// block holding the token's own position writes that row into the cache.  Keys that are not seen: their weights will be 0, and so
// that whatever lies there stays out, their scales too.
template <int D, int G, bool W>
__device__ __forceinline__ void edge_block(const DecodeParams& p, const Int4Task<D, G, W>& d, int b, uint32_t base, int low, int u,
                                           int lane, uint32_t& hide) {
  using R = Int4Record<D>;
  const int bpos = d.block_pos(b);
  const int ntok = min(kBS, d.ctx - bpos);
  const int ov0 = max(bpos, d.nst), nov = p.k_in != nullptr ? bpos + ntok - ov0 : 0;  // this pass's rows: from position ov0 on
  if (nov > 0) {
    const int64_t token0 = d.t - (d.ctx - 1 - ov0);  // the packed token of position ov0
    const int64_t slot = d.ctx - 1 < bpos + kBS ? __ldcg(p.slots + d.t) : -1;
    NewRows<D>::store(p, base, ov0 - bpos, nov, token0, d.g, lane);
    if (slot != -1) write_row<D>(p, base, d.ctx - 1 - bpos, slot, d.g, lane);
  }
  if (ntok < kBS || (W && bpos < low)) {
    auto sees = [&](int key) { return key < ntok && (!W || bpos + key >= low || bpos + key < p.win.sinks); };
    hide |= (sees(lane >> 2) ? 0u : 1u) << (2 * u) | (sees((lane >> 2) + 8) ? 0u : 2u) << (2 * u);
    __syncwarp();
    for (int i = lane; i < kBS * R::GROUPS; i += 32)  // a row's scales are GROUPS words, K's and V's
      if (!sees(i / R::GROUPS)) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + R::SCALES + i * 4), "r"(0) : "memory");
    __syncwarp();
  }
}

// A producer warp: copies the pairs of the streaming warps w with w % NP == which into each warp's own stages, in order.  Two
// lanes serve a streaming warp, one for each record of its pair, and the pairs of one lap around a task go out at once; the first
// producer copies the task's q ahead of them.
template <int D, int G, bool W>
struct Int4Producer {
  using T = DecodeTraits<D, G, kKvInt4>;
  using R = Int4Record<D>;
  const DecodeParams& p;
  const DecodeSmem<D, G, kKvInt4>& sm;
  uint64_t* full;
  uint64_t* empty;
  uint64_t pol;
  int which, lane;
  int w;             // the lane's streaming warp (at or past NW: none)
  int at = 0;        // the warp's stage that its next pair goes to,
  int used = 0;      // and the pairs it has had so far
  uint32_t phase = 1;  // of the stage's emptying (the first passes at once)
  int m = 0, lap = 0;  // of the current task's pairs the first m are copied, the lap's first is `lap`
  int pairs = 0, around = 1, place = 0;  // the current task's (spread); the lane's place in it
  int q_issued = 0;  // tasks whose q is copied

  __device__ Int4Producer(const DecodeParams& p_, const DecodeSmem<D, G, kKvInt4>& sm_, int which_, int lane_)
      : p(p_), sm(sm_), full(sm_.ring_bar), empty(sm_.ring_bar + T::NR), which(which_), lane(lane_), w((lane_ >> 1) * T::NP + which_) {
    pol = dev::l2_policy_evict_first();
  }
  // The pairs of this lap that are not copied yet and below `end`.  False: a wait ran out, and none was copied.
  __device__ bool copy(const typename T::Task& e, int end) {
    const int i = lane & 1, pr = lap + place;
    const bool mine = w < T::NW && place < around && pr >= m && pr < end;
    const int slot = w * T::NRW + at;
    if (!cta_wait_lanes(&empty[mine ? slot : 0], phase, mine, sm.abort, p.err)) return false;
    const int blocks = min(2, e.nb - 2 * pr);
    if (mine && i == 0) dev::mbar_arrive_expect_tx(&full[slot], blocks * R::BYTES);
    __syncwarp();
    if (mine) {
      if (i < blocks)
        dev::bulk_g2s(sm.ring + slot * T::RUN + i * R::BYTES,
                      reinterpret_cast<const char*>(p.cache_k) + ((size_t)e.ids[2 * pr + i] * p.num_kv_heads + (e.rec.y & 0xFF)) * R::BYTES,
                      R::BYTES, &full[slot], pol);
      ++used;
      if (++at == T::NRW) {
        at = 0;
        phase ^= 1;
      }
    }
    m = min(end, lap + around);
    if (m == lap + around) lap = m;
    return true;
  }
  __device__ __forceinline__ void start(const typename T::Task& e) {
    pairs = (e.nb + 1) / 2;
    around = spread<T::NW>(pairs);
    place = dealt<T::NW>(w, e.rot);
  }
  // Before the dependency wait: the first task's leading pairs, wherever nothing that the previous kernel writes can be in
  // their blocks (positions the appended tokens never reach, or rows that are replaced from the inputs anyway).
  __device__ void prologue() {
    const bool got = cta_wait(&sm.qfull[0], 0, sm.abort, p.err);
    if (!__all_sync(0xffffffffu, got)) return;
    const typename T::Task& e = sm.queue[0];
    if (e.rec.x < 0) return;
    start(e);
    if (!p.early) return;
    const Int4Task<D, G, W> d(p, e);
    const int most = min(pairs, around * T::NRW);  // (no stage twice)
    const bool may = lane < most && (p.k_in != nullptr || p.late_wait || d.block_pos(min(2 * lane + 1, e.nb - 1)) + kBS <= e.nst);
    const int lead = __ffs(~__ballot_sync(0xffffffffu, may)) - 1, end = lead < 0 ? 32 : lead;
    while (m < end)
      if (!copy(e, end)) return;
  }
  __device__ void run() {
    for (int k = 0;; ++k) {
      const bool got = cta_wait(&sm.qfull[k % T::QD], (k / T::QD) & 1, sm.abort, p.err);
      if (!__all_sync(0xffffffffu, got)) return;
      const typename T::Task& e = sm.queue[k % T::QD];
      if (e.rec.x < 0) return;
      start(e);
      if (which == 0 && lane == 0) {
        dev::fence_proxy_async_smem();  // the reads of the buffer's previous q (its task is done with) precede this copy
        dev::mbar_arrive_expect_tx(&sm.qbar[k % T::QD], T::QB);
        dev::bulk_g2s(sm.qbuf + (k % T::QD) * T::QB, p.q + ((size_t)e.rec.x * p.num_q_heads + (size_t)(e.rec.y & 0xFF) * G) * D,
                      T::QB, &sm.qbar[k % T::QD], pol);
      }
      if (which == 0) ++q_issued;
      while (m < pairs)
        if (!copy(e, pairs)) return;
      m = lap = 0;
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&sm.qempty[k % T::QD]);
    }
  }
  // The copies must land before the CTA leaves (each wait bounded).
  __device__ void drain() {
    if (w < T::NW && (lane & 1) == 0)
      for (int c = max(0, used - T::NRW); c < used; ++c) dev::mbar_wait(&full[w * T::NRW + c % T::NRW], (c / T::NRW) & 1);
    if (lane == 0)
      for (int k = max(0, q_issued - T::QD); k < q_issued; ++k) dev::mbar_wait(&sm.qbar[k % T::QD], (k / T::QD) & 1);
  }
};

// A streaming warp: of every task the pairs dealt to it, and its share to the combiner warp.
template <int D, int G, bool W>
__device__ __forceinline__ void stream_int4(const DecodeParams& p, const DecodeSmem<D, G, kKvInt4>& sm, int warp, int lane) {
  using T = DecodeTraits<D, G, kKvInt4>;
  using R = Int4Record<D>;
  uint64_t* full = sm.ring_bar;
  uint64_t* empty = sm.ring_bar + T::NR;
  const uint32_t ring = dev::smem_addr(sm.ring);
  int shares = 0;        // shares this warp has handed to the combiner warp
  int at = 0;            // the warp's stage (of NRW) that its next pair comes in
  uint32_t phase = 0;    // and the phase of that stage
  for (int k = 0;; ++k) {
    bool got = cta_wait(&sm.qfull[k % T::QD], (k / T::QD) & 1, sm.abort, p.err);
    if (!__all_sync(0xffffffffu, got)) return;
    const typename T::Task& e = sm.queue[k % T::QD];
    if (e.rec.x < 0) return;
    const Int4Task<D, G, W> d(p, e);
    const int around = spread<T::NW>(d.pairs());
    const int first = dealt<T::NW>(warp, e.rot);                 // the warp's pairs: first, first + around, ...
    const int np = place_pairs(d.pairs(), around, first);
    if (np < 2 && lane == 0) dev::mbar_arrive(&sm.qmid[k % T::QD]);  // the half-way signal (Scheduler): after np / 2 pairs
    if (np > 0) {
      const int low = W ? window_low(d.ctx, p.win.window) : 0;  // the window's first key
      const int b0 = 2 * (first + around * lane);
      const uint32_t edges = __ballot_sync(0xffffffffu, lane < np && (b0 + 1 >= d.nb || d.edge(p, b0, low) || d.edge(p, b0 + 1, low)));
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // references and sums
      float o[T::MT][4];
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

      // q as the MMAs' B operand (k = dims, n = heads; the columns of heads G .. 7 repeat head 0).  K's fragments: lane l's
      // word of a 32-value group is values 8t .. 8t + 7 (t = l % 4), which unpack in pairs (i, i + 4); pairs 0 and 1 are MMA k
      // indices 2t, 2t + 1 and 2t + 8, 2t + 9 of the group's first step, pairs 2 and 3 of its second.  q takes the same
      // order, which leaves every dot product as it is.
      uint32_t qb[T::KS][2];
      got = cta_wait(&sm.qbar[k % T::QD], (k / T::QD) & 1, sm.abort, p.err);
      if (!__all_sync(0xffffffffu, got)) return;
      const uint32_t qs = dev::smem_addr(sm.qbuf) + (k % T::QD) * T::QB + ((lane >> 2) < G ? lane >> 2 : 0) * (D * 2) + (lane & 3) * 16;
#pragma unroll
      for (int g = 0; g < D / 32; ++g) {
        uint32_t x[4];
        dev::lds_words<4>(qs + g * 64, x);
        qb[2 * g][0] = __byte_perm(x[0], x[2], 0x5410);
        qb[2 * g][1] = __byte_perm(x[0], x[2], 0x7632);
        qb[2 * g + 1][0] = __byte_perm(x[1], x[3], 0x5410);
        qb[2 * g + 1][1] = __byte_perm(x[1], x[3], 0x7632);
      }

      for (int i = 0; i < np; ++i) {
        const int slot = warp * T::NRW + at;
        got = cta_wait(&full[slot], phase, sm.abort, p.err);
        if (!__all_sync(0xffffffffu, got)) return;
        uint32_t base[2] = {ring + slot * T::RUN, ring + slot * T::RUN + R::BYTES};
        uint32_t hide = 0;  // bit 2u: key lane / 4 of block u is not seen, bit 2u + 1: key lane / 4 + 8
        if (edges >> i & 1) {  // (rare: what it needs of the task is read again, and no register holds it from pair to pair)
          const typename T::Task& e = sm.queue[k % T::QD];
          const Int4Task<D, G, W> d(p, e);
          const int pr = dealt<T::NW>(warp, e.rot) + spread<T::NW>(d.pairs()) * i, n = min(2, d.nb - 2 * pr);
          const int low = W ? window_low(d.ctx, p.win.window) : 0;
#pragma unroll 1
          for (int u = 0; u < n; ++u) edge_block<D, G, W>(p, d, 2 * pr + u, u == 0 ? base[0] : base[1], low, u, lane, hide);
          if (n < 2) {  // an odd last block is its own twin, of which nothing is seen
            base[1] = base[0];
            hide |= 12u;
          }
          dev::fence_proxy_async_smem();  // generic writes precede the stage's next bulk copy
        }
        attend_pair<D>(base, hide, qb, p.scale_log2, lane, m0, m1, l0, l1, o);
        __syncwarp();  // every lane has read the stage
        if (lane == 0) dev::mbar_arrive(&empty[slot]);
        if (++at == T::NRW) {
          at = 0;
          phase ^= 1;
        }
        if (i + 1 == np / 2 && lane == 0) dev::mbar_arrive(&sm.qmid[k % T::QD]);
      }

      // ---- hand this warp's share of the split to the combiner warp ----
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, m);
        l1 += __shfl_xor_sync(0xffffffffu, l1, m);
      }
      if (shares > 0) {  // the slot is free once the combiner warp has taken the previous share
        got = cta_wait(&sm.share_empty[warp], (shares - 1) & 1, sm.abort, p.err);
        if (!__all_sync(0xffffffffu, got)) return;
      }
      const int hg = lane & 3;
      if (hg < T::LG) {
        float* my_o = sm.sh_o + warp * T::OV * T::SHL;
        float2* my_ml = sm.sh_ml + warp * kHeadsTile;
        const int ci = (lane >> 2) * T::LG + hg;
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt)
          reinterpret_cast<float4*>(my_o)[mt * T::SHL + ci] = make_float4(o[mt][0], o[mt][1], o[mt][2], o[mt][3]);
        if (lane < T::LG) {
          my_ml[2 * lane] = make_float2(m0, l0);
          my_ml[2 * lane + 1] = make_float2(m1, l1);
        }
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&sm.share_full[warp]);
      ++shares;
    }
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(&sm.qempty[k % T::QD]);  // done with the task's queue entry
  }
}

// Merges a token whose splits are all counted, from L2, whichever CTA it is: lane i has the weights of split i (at most 32), and
// the values are summed in order, two splits' loads at a time and the first ahead of the weights.  (At the end of a launch a CTA
// may have several of these one behind another, each 4 us when the weights came with every group of values.)
template <int D, int G>
__device__ __forceinline__ void merge_int4(const DecodeParams& p, int tg, int nsplit, int lane) {
  static_assert(kFusedMergeSplits <= 32, "a lane a split");
  constexpr int NG = G * D / 4, EG = (NG + 31) / 32;  // groups of 4 consecutive dims of one head; of them a lane's
  constexpr int CH = EG <= 6 ? EG : 4;                // of which so many at a time
  const size_t sb = (size_t)tg * p.max_splits;
  const int t = tg / p.num_kv_heads, g = tg % p.num_kv_heads;
  __half* out = p.out + ((size_t)t * p.num_q_heads + (size_t)g * G) * D;
  float2 ml[G];
#pragma unroll
  for (int h = 0; h < G; ++h)
    ml[h] = lane < nsplit ? __ldcg(p.part_ml + (sb + lane) * kHeadsTile + h) : make_float2(-INFINITY, 0.f);
  float weight[G];
#pragma unroll
  for (int j0 = 0; j0 < EG; j0 += CH) {
    float4 acc[CH], o[2][CH];
    auto load = [&](int s0) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < CH; ++j) {  // (past the last split the last, past the last group the lane's first: unused)
          const int e4 = lane + 32 * (j0 + j), s = min(s0 + u, nsplit - 1);
          o[u][j] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (sb + s) * kHeadsTile * D) + (e4 < NG ? e4 : lane % NG));
        }
    };
    load(0);
    if (j0 == 0) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float M = ml[h].x;
        for (int i = 1; i < nsplit; i <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
        const float f = lane < nsplit ? dev::ex2_approx(ml[h].x - M) : 0.f;
        float L = ml[h].y * f;
        for (int i = 1; i < nsplit; i <<= 1) L += __shfl_xor_sync(0xffffffffu, L, i);
        weight[h] = f / L;
      }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = 0;;) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (s0 + u >= nsplit) break;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int h = (j0 + j) * 128 / D, h1 = h + 1 < G ? h + 1 : h;  // the group's head (d 64: of the lower lanes)
          if (h >= G) continue;
          float w = __shfl_sync(0xffffffffu, weight[h], s0 + u);
          if constexpr (D == 64) {
            const float w1 = __shfl_sync(0xffffffffu, weight[h1], s0 + u);
            if (lane >= 16) w = w1;
          }
          acc[j].x = fmaf(o[u][j].x, w, acc[j].x);
          acc[j].y = fmaf(o[u][j].y, w, acc[j].y);
          acc[j].z = fmaf(o[u][j].z, w, acc[j].z);
          acc[j].w = fmaf(o[u][j].w, w, acc[j].w);
        }
      }
      s0 += 2;
      if (s0 >= nsplit) break;
      load(s0);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int e4 = lane + 32 * (j0 + j);
      if (e4 < NG)
        *reinterpret_cast<uint2*>(out + 4 * e4) =
            make_uint2(dev::as_word(__floats2half2_rn(acc[j].x, acc[j].y)), dev::as_word(__floats2half2_rn(acc[j].z, acc[j].w)));
    }
  }
}

// The combiner warp: folds a task's shares and writes the token's output or the split's partial, which it counts on the token;
// where the count (looked at when the next task is in hand) completes the token, it merges it.
// A warp beside streaming warps gets about one instruction in ten cycles and a spilled register costs it a trip to L2 (shared
// memory leaves no L1): the fold keeps few registers, and nothing of a task outlives it but the count.
template <int D, int G, bool W>
__device__ __forceinline__ void combine_int4(const DecodeParams& p, const DecodeSmem<D, G, kKvInt4>& sm, int lane) {
  using T = DecodeTraits<D, G, kKvInt4>;
  uint32_t taken = 0;  // bit w: parity of the shares taken from streaming warp w so far
  int last_tg = -1, last_ns = 0, prev = 0;  // the partial counted last, and (lane 0) the count before it
  const int hg = lane & 3;
  const bool real = hg < T::LG;  // this lane's fragment columns hold real heads
  const int ci = (lane >> 2) * T::LG + hg;
  for (int k = 0;; ++k) {
    const bool got = cta_wait(&sm.qfull[k % T::QD], (k / T::QD) & 1, sm.abort, p.err);
    if (!__all_sync(0xffffffffu, got)) return;
    const typename T::Task* e = &sm.queue[k % T::QD];
    const int4 rec = e->rec;
    const int nb = e->nb, rot = e->rot;
    __syncwarp();
    if (last_tg >= 0 && __shfl_sync(0xffffffffu, prev, 0) == last_ns - 1) {
      if (lane == 0) p.merge_cnt[last_tg] = 0;  // ready for the next launch on this plan
      __syncwarp();
      merge_int4<D, G>(p, last_tg, last_ns, lane);
    }
    last_tg = -1;
    if (rec.x < 0) return;
    if (lane == 0) dev::mbar_arrive(&sm.qempty[k % T::QD]);
    const int t = rec.x, g = rec.y & 0xFF, s = rec.y >> 8, ctx = rec.w;
    const int size = split_size<W>(p, ctx);
    const int nsplit = (token_blocks<W>(p, ctx).n + size - 1) / size;
    const int tg = t * p.num_kv_heads + g;
    // ---- the shares, a lane for each (one after another, shares long there took 0.2 us apiece) ----
    const int around = spread<T::NW>((nb + 1) / 2);
    auto warp_at = [&](int place) { return place + rot < T::NW ? place + rot : place + rot - T::NW; };
    const bool mine = lane < T::NW && dealt<T::NW>(lane, rot) < around;
    if (!cta_wait_lanes(&sm.share_full[mine ? lane : 0], (taken >> lane) & 1, mine, sm.abort, p.err)) return;
    const uint32_t there = __ballot_sync(0xffffffffu, mine);
    taken ^= there;
    // ---- references, sums and factors: lane 4 i + hg has the two heads of places i and i + 8 (one tree, whatever rot is) ----
    float4 ml[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int place = (lane >> 2) + 8 * i;
      ml[i] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      if (real && place < around) ml[i] = *reinterpret_cast<const float4*>(sm.sh_ml + warp_at(place) * kHeadsTile + 2 * hg);
    }
    float M0 = fmaxf(ml[0].x, ml[1].x), M1 = fmaxf(ml[0].z, ml[1].z), L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      M0 = fmaxf(M0, __shfl_xor_sync(0xffffffffu, M0, o));
      M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, o));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int place = (lane >> 2) + 8 * i;
      if (real && place < around) {
        ml[i].x = dev::ex2_approx(ml[i].x - M0);
        ml[i].z = dev::ex2_approx(ml[i].z - M1);
        L0 = fmaf(ml[i].y, ml[i].x, L0);
        L1 = fmaf(ml[i].w, ml[i].z, L1);
        *reinterpret_cast<float4*>(sm.sh_ml + warp_at(place) * kHeadsTile + 2 * hg) = ml[i];
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      L0 += __shfl_xor_sync(0xffffffffu, L0, o);
      L1 += __shfl_xor_sync(0xffffffffu, L1, o);
    }
    __syncwarp();
    // ---- the values, four fragments at a time, two to an instruction.  A lane's are fours of consecutive dims ----
    if (real) {
      constexpr int FG = 4, B = 2;
      static_assert(T::MT % FG == 0, "fragments");
      const float i0 = 1.f / L0, i1 = 1.f / L1;
      const size_t pidx = (size_t)tg * p.max_splits + s;
      __half* out = p.out + ((size_t)t * p.num_q_heads + (size_t)g * G) * D;
      float* part = p.part_o + pidx * kHeadsTile * D;
#pragma unroll 1
      for (int m0 = 0; m0 < T::MT; m0 += FG) {
        float2 x[FG][2];
#pragma unroll
        for (int i = 0; i < FG; ++i) x[i][0] = x[i][1] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int first = 0; first < around; first += B) {  // past the last share the first with weight 0
          float4 v[B][FG];
          float2 f[B];
#pragma unroll
          for (int u = 0; u < B; ++u) {
            const bool in = first + u < around;
            const int w = warp_at(in ? first + u : 0);
            const float4 fu = *reinterpret_cast<const float4*>(sm.sh_ml + w * kHeadsTile + 2 * hg);
            f[u] = in ? make_float2(fu.x, fu.z) : make_float2(0.f, 0.f);
            const float4* so = reinterpret_cast<const float4*>(sm.sh_o + w * T::OV * T::SHL) + m0 * T::SHL + ci;
#pragma unroll
            for (int i = 0; i < FG; ++i) v[u][i] = so[i * T::SHL];
          }
#pragma unroll
          for (int u = 0; u < B; ++u)
#pragma unroll
            for (int i = 0; i < FG; ++i) {
              x[i][0] = dev::fma2(make_float2(v[u][i].x, v[u][i].y), f[u], x[i][0]);
              x[i][1] = dev::fma2(make_float2(v[u][i].z, v[u][i].w), f[u], x[i][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < FG; i += 2)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int head = 2 * hg + h, at = head * D + 16 * (m0 + i) + 4 * (lane >> 2);
            if (head >= G) continue;
            const float4 y = h ? make_float4(x[i][0].y, x[i][1].y, x[i + 1][0].y, x[i + 1][1].y)
                               : make_float4(x[i][0].x, x[i][1].x, x[i + 1][0].x, x[i + 1][1].x);
            if (nsplit == 1) {
              const float il = h ? i1 : i0;
              *reinterpret_cast<uint2*>(out + at) =
                  make_uint2(dev::as_word(__floats2half2_rn(y.x * il, y.y * il)), dev::as_word(__floats2half2_rn(y.z * il, y.w * il)));
            } else {
              *reinterpret_cast<float4*>(part + at) = y;
            }
          }
      }
      if (nsplit > 1 && lane < T::LG) {
        if (2 * lane < G) p.part_ml[pidx * kHeadsTile + 2 * lane] = make_float2(M0, L0);
        if (2 * lane + 1 < G) p.part_ml[pidx * kHeadsTile + 2 * lane + 1] = make_float2(M1, L1);
      }
    }
    __syncwarp();
    if (there >> lane & 1) dev::mbar_arrive(&sm.share_empty[lane]);
    if (nsplit > 1 && nsplit <= kFusedMergeSplits) {
      last_tg = tg;
      last_ns = nsplit;
      if (lane == 0) prev = dev::atom_add_acq_rel_gpu(p.merge_cnt + tg, 1);  // (the warp's stores precede it)
    }
  }
}

template <int D, int G, bool W>
__global__ void __launch_bounds__(DecodeTraits<D, G, kKvInt4>::NTHREADS, 1) decode_int4_kernel(const __grid_constant__ DecodeParams p) {
  using T = DecodeTraits<D, G, kKvInt4>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const DecodeSmem<D, G, kKvInt4> sm(smem);
  // warps: streaming 0 .. NW - 1, combiner, scheduler, producers
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // set-up that reads nothing written by earlier kernels runs before the dependency wait
  if (threadIdx.x == 0) {
    for (int i = 0; i < T::RB; ++i) dev::mbar_init(&sm.ring_bar[i], 1);
    for (int i = 0; i < T::NW; ++i) {
      dev::mbar_init(&sm.share_full[i], 1);
      dev::mbar_init(&sm.share_empty[i], 1);
    }
    for (int i = 0; i < T::QD; ++i) {
      dev::mbar_init(&sm.qfull[i], 1);
      dev::mbar_init(&sm.qempty[i], T::NW + 1 + T::NP);  // the streaming warps, the combiner and the producers
      dev::mbar_init(&sm.qmid[i], T::NW);       // the streaming warps
    }
    for (int i = 0; i < T::NQ; ++i) dev::mbar_init(&sm.qbar[i], 1);
    *sm.abort = 0;
    dev::fence_mbar_init();
  }
  __syncwarp();
  __syncthreads();
  // What is read before the dependency wait: see decode_kernel (decode.cuh).
  const bool producer = warp > T::NW + 1;
  Int4Producer<D, G, W> pr(p, sm, warp - T::NW - 2, lane);
  Scheduler<D, G, kKvInt4, W> sch(p, sm, lane);
  if (warp == T::NW + 1) sch.prologue();
  if (producer) pr.prologue();
  __syncwarp();
  if (!p.late_wait) dev::griddep_wait();
  dev::griddep_launch_dependents();
  // one CTA-uniform decision (a racing error-word update must not split the CTA)
  int pz = 0;
  if (threadIdx.x == 0) pz = dev::pool_poisoned(p.err) ? 1 : 0;
  __syncwarp();
  const bool poisoned = __syncthreads_or(pz);
  if (producer) {
    if (!poisoned) pr.run();
    __syncwarp();
    pr.drain();
  } else if (!poisoned) {
    if (warp < T::NW) stream_int4<D, G, W>(p, sm, warp, lane);
    else if (warp == T::NW) combine_int4<D, G, W>(p, sm, lane);
    else sch.run();
  }
  // The last CTA out resets the task counter for the next launch on this plan (no fence: decode_kernel).
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (atomicAdd(&p.hdr->done, 1) == (int)gridDim.x - 1) {
      p.hdr->work = 0;
      p.hdr->done = 0;
    }
  }
  if (p.late_wait) dev::griddep_wait();  // complete only after the prefill kernel ahead of it
}

template <int D, int G, bool W>
static cudaError_t launch_int4(const DecodeParams& p, pkv_pool* pool, int64_t max_tasks, cudaStream_t stream) {
  using T = DecodeTraits<D, G, kKvInt4>;
  const cudaError_t e = prepare_kernel(pool, decode_int4_kernel<D, G, W>, T::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(pool->num_sms, max_tasks));  // persistent: one CTA per SM
  return launch_pdl(decode_int4_kernel<D, G, W>, dim3((unsigned)grid), dim3(T::NTHREADS), T::SMEM, stream, p);
}

template <bool W>
static cudaError_t launch_int4_shape(int head_dim, int group, const DecodeParams& p, pkv_pool* pool, int64_t max_tasks,
                                     cudaStream_t stream) {
  switch (head_dim * 16 + group) {
    case 64 * 16 + 1: return launch_int4<64, 1, W>(p, pool, max_tasks, stream);
    case 64 * 16 + 2: return launch_int4<64, 2, W>(p, pool, max_tasks, stream);
    case 64 * 16 + 4: return launch_int4<64, 4, W>(p, pool, max_tasks, stream);
    case 64 * 16 + 6: return launch_int4<64, 6, W>(p, pool, max_tasks, stream);
    case 64 * 16 + 8: return launch_int4<64, 8, W>(p, pool, max_tasks, stream);
    case 128 * 16 + 1: return launch_int4<128, 1, W>(p, pool, max_tasks, stream);
    case 128 * 16 + 2: return launch_int4<128, 2, W>(p, pool, max_tasks, stream);
    case 128 * 16 + 4: return launch_int4<128, 4, W>(p, pool, max_tasks, stream);
    case 128 * 16 + 6: return launch_int4<128, 6, W>(p, pool, max_tasks, stream);
    case 128 * 16 + 8: return launch_int4<128, 8, W>(p, pool, max_tasks, stream);
    case 256 * 16 + 1: return launch_int4<256, 1, W>(p, pool, max_tasks, stream);
    case 256 * 16 + 2: return launch_int4<256, 2, W>(p, pool, max_tasks, stream);
    case 256 * 16 + 4: return launch_int4<256, 4, W>(p, pool, max_tasks, stream);
    case 256 * 16 + 6: return launch_int4<256, 6, W>(p, pool, max_tasks, stream);
    case 256 * 16 + 8: return launch_int4<256, 8, W>(p, pool, max_tasks, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
