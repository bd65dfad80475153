// Rotary positions, fused with the append; the same with a norm of every query and key head in front.
//
// Pair i of a head turns by position * f_i: a' = a cos - b sin, b' = b cos + a sin.  The pages have no
// counterpart; the keys land in their slots as kv_append stores them ("Continuous Batching Is Not a Bigger Batch",
// opening section and "The allocator is the other half").
//
// Angles: the position reaches millions and cos needs it modulo a turn, where a 32-bit product has no bits left.  So
// f_i / (2 pi) is a 64-bit binary fraction of a turn; position times it, wrapping modulo 2^64, is that fraction's angle
// modulo a turn, exactly, and its upper half (a signed 32-bit fraction of a turn) goes to sincospif.  The fraction comes
// from a 64-bit float: 53 bits, off by less than 2^-53 of a turn for frequencies up to 1.
// No 64-bit floating point on the device.
//
// Norms: y = x / sqrt(mean(x^2) + eps) * (offset + w) over a head's head_dim values, all in fp32: the mean square, the
// product and the rotation behind it, with one rounding to fp16 at the end.
//
// Bound by memory: q, k and v read once, q_out and the slots written once.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "int4.cuh"
#include "pkv_internal.cuh"

constexpr int kMaxPairs = 128;

struct pkv_rope {
  pkv_rope_config cfg;
  double freq[kMaxPairs];     // radians a token
  uint64_t turn[kMaxPairs];   // the same as a fraction of a turn times 2^64
};

namespace pkv {

namespace {

struct RopeTurns {
  uint64_t turn[kMaxPairs];
};

struct RopeParams {
  const __half* q;
  const __half* k;
  const __half* v;
  __half* q_out;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;
  const int64_t* slots;
  unsigned char* cache_k;   // this layer's K pool: fp16 rows, or codes
  unsigned char* cache_v;
  unsigned char* scales;
  int64_t num_slots;
  int num_tokens, num_q_heads, num_kv_heads;
  int tokens;               // per CTA
  int rot_dim;
  float out_scale;
  int32_t* err;
  // Norms: a head's weights, [head_dim]; null: its heads are not normalised.
  const __half* q_weight;
  const __half* k_weight;
  float eps, weight_offset;
};

constexpr int kThreads = 128;
constexpr int kMaxTokens = 4;  // per CTA

__device__ __forceinline__ uint4 ld16(const __half* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// One rotated pair of fp16 vectors of 8 values: pair j is (a_j, b_j).
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(pa + j)), y = __half22float2(*reinterpret_cast<__half2*>(pb + j));
    const __half2 u = __floats2half2_rn(x.x * c[2 * j] - y.x * s[2 * j], x.y * c[2 * j + 1] - y.y * s[2 * j + 1]);
    const __half2 w = __floats2half2_rn(y.x * c[2 * j] + x.x * s[2 * j], y.y * c[2 * j + 1] + x.y * s[2 * j + 1]);
    pa[j] = *reinterpret_cast<const uint32_t*>(&u);
    pb[j] = *reinterpret_cast<const uint32_t*>(&w);
  }
}
// The same with the pairs side by side: (a_0, a_1), (a_2, a_3), .., then b's.
__device__ __forceinline__ void rotate8_interleaved(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
  uint32_t* w[2] = {reinterpret_cast<uint32_t*>(&a), reinterpret_cast<uint32_t*>(&b)};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t& r = w[j >> 2][j & 3];
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&r));
    const __half2 u = __floats2half2_rn(x.x * c[j] - x.y * s[j], x.y * c[j] + x.x * s[j]);
    r = *reinterpret_cast<const uint32_t*>(&u);
  }
}

// A CTA rotates `tokens` tokens.  Every angle is computed once, by one thread, into shared memory (a sincospif costs
// more than the loads and stores of a chunk: with the 8 angles of a 16-value piece computed where they were used, once
// for every few heads, 8192 tokens took 15 to 21 us).  The unit of the rest is an item: 16 values of a q or KV head (two
// 16-byte chunks that hold 8 whole pairs, or 16 values past the rotated part; of a KV head the key's and the value's).
// A thread loads its first items before it computes its angles, so that neither waits for the other.  On a 4-bit cache a
// scale's 32 values are four 8-value chunks of up to four items: the chunks' largest magnitudes meet in shared memory.
template <int D, int KV, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p, const __grid_constant__ RopeTurns turns) {
  constexpr int PC = D / 16;  // items per head: a power of two within a warp
  constexpr int U = 2;        // items in flight a thread
  static_assert(kThreads % PC == 0 && 32 % PC == 0, "a thread's items are one piece of different heads");
  __shared__ uint4 chunk_amax[KV == PKV_KV_INT4 ? kThreads / 2 : 1];  // [thread's head][chunk] largest magnitude
  // (cos, sin) of pairs 2j and 2j + 1 of a token's rotated 16-value piece pc at [token][j][pc]: consecutive lanes read
  // consecutive 16 bytes
  __shared__ float4 angle[kMaxTokens][4][PC];
  const int half = p.rot_dim / 2, pieces = p.rot_dim / 16;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int n = (int)min((int64_t)p.tokens, p.num_tokens - t0);
  const int heads = p.num_q_heads + p.num_kv_heads;  // q heads, then KV heads
  const uint32_t per = heads * PC, items = n * per;
  dev::griddep_wait();
  dev::griddep_launch_dependents();
  for (uint32_t i0 = 0; i0 < items; i0 += U * kThreads) {  // the same number of rounds in every thread
    uint4 a[U], b[U], va[U], vb[U];
    int64_t slot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads + threadIdx.x, tb = i / per;
      const int h = (int)((i - tb * per) / PC), pc = (int)(i % PC), g = h - p.num_q_heads;
      const int64_t t = t0 + tb;
      const int c0 = !INTER && pc < pieces ? pc : 2 * pc, c1 = !INTER && pc < pieces ? pc + half / 8 : 2 * pc + 1;
      a[u] = b[u] = va[u] = vb[u] = make_uint4(0, 0, 0, 0);
      slot[u] = -1;
      if (i >= items) continue;
      if (g < 0) {  // plain loads: q_out may be q
        const uint4* src = reinterpret_cast<const uint4*>(p.q + t * p.q_stride + (int64_t)h * D);
        a[u] = src[c0];
        b[u] = src[c1];
      } else {
        const __half* ks = p.k + t * p.k_stride + (int64_t)g * D;
        const __half* vs = p.v + t * p.v_stride + (int64_t)g * D;
        slot[u] = __ldg(p.slots + t);
        a[u] = ld16(ks + 8 * c0);
        b[u] = ld16(ks + 8 * c1);
        va[u] = ld16(vs + 16 * pc);
        vb[u] = ld16(vs + 16 * pc + 8);
      }
    }
    if (i0 == 0) {
      for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int tb = i / half, k = i - tb * half;  // pair k: of piece k / 8, its pair k % 8
        const uint64_t pos = (uint64_t)(int64_t)__ldg(p.positions + t0 + tb);
        const int32_t turn = (int32_t)((pos * turns.turn[k]) >> 32);
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        reinterpret_cast<float2*>(&angle[tb][(k & 7) >> 1][k >> 3])[k & 1] = make_float2(c * p.out_scale, s * p.out_scale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads + threadIdx.x, tb = i / per;
      const int h = (int)((i - tb * per) / PC), pc = (int)(i % PC), g = h - p.num_q_heads;
      const int64_t t = t0 + tb;
      const bool in = i < items, rot = pc < pieces;
      const int c0 = !INTER && rot ? pc : 2 * pc, c1 = !INTER && rot ? pc + half / 8 : 2 * pc + 1;
      const bool kv = in && g >= 0 && slot[u] >= 0 && slot[u] < p.num_slots;
      if (in && g == 0 && pc == 0 && slot[u] != -1 && !kv) dev::set_error(p.err, PKV_DEVERR_SLOT_RANGE);
      if (in && rot) {
        float cs[8], sn[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 x = angle[tb][j][pc];
          cs[2 * j] = x.x;
          sn[2 * j] = x.y;
          cs[2 * j + 1] = x.z;
          sn[2 * j + 1] = x.w;
        }
        if constexpr (INTER) rotate8_interleaved(a[u], b[u], cs, sn); else rotate8(a[u], b[u], cs, sn);
      }
      if (in && g < 0) {
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + (t * p.num_q_heads + h) * D);
        dst[c0] = a[u];
        dst[c1] = b[u];
      }
      const int64_t row = kv ? ((slot[u] >> 4) * p.num_kv_heads + g) * 16 + (slot[u] & 15) : 0;
      if constexpr (KV == PKV_KV_INT4) {
        uint32_t* amax = reinterpret_cast<uint32_t*>(chunk_amax) + 2 * (threadIdx.x - pc);  // this head's chunks
        amax[c0] = dev::f16x8_amax_bits(a[u]);
        amax[c1] = dev::f16x8_amax_bits(b[u]);
        const uint32_t av = dev::row_amax_bits<2>(max(dev::f16x8_amax_bits(va[u]), dev::f16x8_amax_bits(vb[u])));
        __syncwarp();
        const uint4 m0 = reinterpret_cast<const uint4*>(amax)[c0 >> 2], m1 = reinterpret_cast<const uint4*>(amax)[c1 >> 2];
        __syncwarp();  // read before the next item's go over them
        if (kv) {
          using R = Int4Record<D>;
          const __half s0 = dev::int4_scale(max(max(m0.x, m0.y), max(m0.z, m0.w)));
          const __half s1 = dev::int4_scale(max(max(m1.x, m1.y), max(m1.z, m1.w)));
          const __half sv = dev::int4_scale(av);
          unsigned char* rec = p.cache_k + ((slot[u] >> 4) * p.num_kv_heads + g) * R::BYTES;
          const int r = (int)(slot[u] & 15);
          *reinterpret_cast<uint32_t*>(rec + R::code_at(0, r, c0)) = dev::int4_encode8(a[u], s0);
          *reinterpret_cast<uint32_t*>(rec + R::code_at(0, r, c1)) = dev::int4_encode8(b[u], s1);
          *reinterpret_cast<uint2*>(rec + R::code_at(1, r, 2 * pc)) =
              make_uint2(dev::int4_encode8(va[u], sv), dev::int4_encode8(vb[u], sv));
          if ((c0 & 3) == 0) *reinterpret_cast<__half*>(rec + R::scale_at(0, r, c0)) = s0;
          if ((c1 & 3) == 0) *reinterpret_cast<__half*>(rec + R::scale_at(0, r, c1)) = s1;
          if ((pc & 1) == 0) *reinterpret_cast<__half*>(rec + R::scale_at(1, r, 2 * pc)) = sv;
        }
      } else if constexpr (KV == PKV_KV_E4M3) {
        // a row's PC lanes are consecutive and lane-aligned; every lane of the warp takes part
        const uint32_t ak = dev::row_amax_bits<PC>(max(dev::f16x8_amax_bits(a[u]), dev::f16x8_amax_bits(b[u])));
        const uint32_t av = dev::row_amax_bits<PC>(max(dev::f16x8_amax_bits(va[u]), dev::f16x8_amax_bits(vb[u])));
        if (kv) {
          const int sbk = dev::e4m3_scale_byte(ak), sbv = dev::e4m3_scale_byte(av);
          uint2* dk = reinterpret_cast<uint2*>(p.cache_k + row * D);
          uint2* dv = reinterpret_cast<uint2*>(p.cache_v + row * D);
          dk[c0] = dev::e4m3_encode8(a[u], sbk);
          dk[c1] = dev::e4m3_encode8(b[u], sbk);
          dv[2 * pc] = dev::e4m3_encode8(va[u], sbv);
          dv[2 * pc + 1] = dev::e4m3_encode8(vb[u], sbv);
          if (pc == 0) {
            unsigned char* rec = p.scales + ((slot[u] >> 4) * p.num_kv_heads + g) * 32;
            rec[slot[u] & 15] = (unsigned char)sbk;
            rec[16 + (slot[u] & 15)] = (unsigned char)sbv;
          }
        }
      } else if (kv) {
        uint4* dk = reinterpret_cast<uint4*>(p.cache_k + row * (2 * D));
        uint4* dv = reinterpret_cast<uint4*>(p.cache_v + row * (2 * D));
        dk[c0] = a[u];
        dk[c1] = b[u];
        dv[2 * pc] = va[u];
        dv[2 * pc + 1] = vb[u];
      }
    }
  }
}

// ---- with norms ----

__device__ __forceinline__ void to_floats(const uint4& r, float2 (&x)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
}
__device__ __forceinline__ uint4 to_halves(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __floats2half2_rn(x[j].x, x[j].y);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The norms' kernel.  Its unit is a step: a warp's 32 lanes hold 512 values of a token, 16 each (the pieces of the items
// above), of whole q heads, of whole key heads or of whole value heads, so that what a step does is the same for the warp.
// The steps of all tokens are dealt out in equal runs, one to a warp of the whole grid; a warp goes through its run with the
// next two steps' loads under way and the next token's position and slot at hand, computes a token's angles when it comes to it
// (its lanes share them out) and keeps those of its piece in registers; the weights, offset added, lie in shared memory.
// One token of 12 / 2 heads at d 128: 2.0 us in a replayed graph, a launch; 8192 such tokens (67 MB): 17.1 us, on an 8-bit
// cache 18.5, on a 4-bit one 20.1.  Bound by instructions: 264 a step with its share of the angles, 2.4 issued a cycle and SM,
// while the rotation alone takes 13.1 us for the same bytes (their floor is 10.1).  (The items above with a norm in them, all
// heads' weights in registers: 21.5 us.  A step has one weight and no lane of another kind, and its arithmetic is two values
// to an instruction.)
template <int D>
struct NormSteps {
  static constexpr int PC = D / 16, HP = 32 / PC;  // lanes of a head, heads of a step
  int q, kv;                                       // steps of a token's queries, and of its keys (and of its values)
  __host__ __device__ NormSteps(int q_heads, int kv_heads) : q((q_heads + HP - 1) / HP), kv((kv_heads + HP - 1) / HP) {}
  __host__ __device__ int all() const { return q + 2 * kv; }
};

// CTAs per SM, 80 registers a thread.  8192 tokens took 19.7 us with four, 17.8 with five, 17.1 with six, 19.2 with eight (which
// spill); with one step ahead instead of two 18.5 with six, 17.3 with eight; with four ahead 17.4 with four or five.
constexpr int kNormCtas = 6;

template <int D, int KV, bool INTER>
__global__ void __launch_bounds__(kThreads, kNormCtas) norm_rope_append_kernel(const RopeParams p, const __grid_constant__ RopeTurns turns) {
  using S = NormSteps<D>;
  constexpr int PC = S::PC, HP = S::HP, WARPS = kThreads / 32;
  __shared__ uint4 chunk_amax[KV == PKV_KV_INT4 ? kThreads / 2 : 1];  // [thread's head][chunk] largest magnitude
  __shared__ uint64_t turn[D / 2];
  __shared__ float4 weight[2][4][PC];     // q's and k's: values 4 j .. 4 j + 3 of a lane's 16 at [j][lane's piece]
  __shared__ float4 angle[WARPS][4][PC];  // (cos, cos, sin, sin) of a piece's pairs 2 j and 2 j + 1
  const int half = p.rot_dim / 2, pieces = p.rot_dim / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pc = lane % PC, hl = lane / PC;
  const bool rot = pc < pieces;
  const int c0 = !INTER && rot ? pc : 2 * pc, c1 = !INTER && rot ? pc + half / 8 : 2 * pc + 1;  // the lane's two 8-value chunks
  const S steps(p.num_q_heads, p.num_kv_heads);
  const int64_t total = (int64_t)p.num_tokens * steps.all(), warps = (int64_t)gridDim.x * WARPS, me = (int64_t)blockIdx.x * WARPS + warp;
  const int64_t begin = total * me / warps;
  const int count = (int)(total * (me + 1) / warps - begin);
  for (int k = threadIdx.x; k < half; k += kThreads) turn[k] = turns.turn[k];
  dev::griddep_wait();
  dev::griddep_launch_dependents();

  struct Step {
    int64_t t;
    int s;
  };
  auto advance = [&](Step& x) {
    if (++x.s == steps.all()) {
      x.s = 0;
      ++x.t;
    }
  };
  auto load = [&](const Step& x, bool there, uint4& a, uint4& b) {
    const bool q = x.s < steps.q, v = x.s >= steps.q + steps.kv;
    const int h = (q ? x.s : v ? x.s - steps.q - steps.kv : x.s - steps.q) * HP + hl;
    a = b = make_uint4(0, 0, 0, 0);
    if (!there || h >= (q ? p.num_q_heads : p.num_kv_heads)) return;
    const uint4* src = reinterpret_cast<const uint4*>((q ? p.q + x.t * p.q_stride : v ? p.v + x.t * p.v_stride : p.k + x.t * p.k_stride) +
                                                      (int64_t)h * D);
    a = src[c0];  // plain loads: q_out may be q
    b = src[c1];
  };
  Step cur{begin / steps.all(), 0}, ahead;
  cur.s = (int)(begin - cur.t * steps.all());
  ahead = cur;
  uint4 a[2], b[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    load(ahead, u < count, a[u], b[u]);
    advance(ahead);
  }
  const int64_t last = p.num_tokens - 1;
  int64_t slot = count > 0 ? __ldg(p.slots + cur.t) : -1, next_slot = -1;
  int pos = count > 0 && half > 0 ? __ldg(p.positions + cur.t) : 0, next_pos = 0;
  for (int i = threadIdx.x; i < 8 * PC; i += kThreads) {  // both weights, four values at a time
    const int k = i / (4 * PC), j = i / PC % 4, pi = i % PC;
    const __half* w = k ? p.k_weight : p.q_weight;
    const int chunk = !INTER && pi < pieces ? pi + (j >> 1) * (half / 8) : 2 * pi + (j >> 1);
    if (w == nullptr) continue;
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(w + 8 * chunk + 4 * (j & 1)));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&x.x)), hi = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
    weight[k][j][pi] = make_float4(p.weight_offset + lo.x, p.weight_offset + lo.y, p.weight_offset + hi.x, p.weight_offset + hi.y);
  }
  __syncthreads();

  float2 cs[4], sn[4];
  bool fresh = true;  // the current token's angles are still to be computed
  auto process = [&](uint4& a, uint4& b) {
    if (fresh) {
      fresh = false;
      if (cur.t < last) {
        next_slot = __ldg(p.slots + cur.t + 1);
        if (half > 0) next_pos = __ldg(p.positions + cur.t + 1);
      }
      for (int k = lane; k < half; k += 32) {  // pair k: of piece k / 8, its pair k % 8
        float s, c;
        sincospif((float)(int32_t)(((uint64_t)(int64_t)pos * turn[k]) >> 32) * 0x1p-31f, &s, &c);
        float* at = reinterpret_cast<float*>(&angle[warp][(k & 7) >> 1][k >> 3]) + (k & 1);
        at[0] = c * p.out_scale;
        at[2] = s * p.out_scale;
      }
      __syncwarp();
      if (rot) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 x = angle[warp][j][pc];
          cs[j] = make_float2(x.x, x.y);
          sn[j] = make_float2(x.z, x.w);
        }
      }
      __syncwarp();
    }
    const bool q = cur.s < steps.q, v = cur.s >= steps.q + steps.kv;
    const int h = (q ? cur.s : v ? cur.s - steps.q - steps.kv : cur.s - steps.q) * HP + hl;
    const bool in = h < (q ? p.num_q_heads : p.num_kv_heads);
    if (!v) {
      float2 xa[4], xb[4];
      to_floats(a, xa);
      to_floats(b, xb);
      if (q ? p.q_weight != nullptr : p.k_weight != nullptr) {
        float2 s2 = dev::mul2(xa[0], xa[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) s2 = dev::fma2(xa[j], xa[j], s2);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = dev::fma2(xb[j], xb[j], s2);
        float sum = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < PC; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(fmaf(sum, 1.f / D, p.eps));  // (within 2^-22 of it)
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = weight[q ? 0 : 1][j][pc];
          float2* x = j < 2 ? xa + 2 * j : xb + 2 * j - 4;
          x[0] = dev::mul2(x[0], dev::mul2(r2, make_float2(w.x, w.y)));
          x[1] = dev::mul2(x[1], dev::mul2(r2, make_float2(w.z, w.w)));
        }
      }
      if (rot) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (INTER) {  // pairs 2 j and 2 j + 1 side by side
            float2* x = j < 2 ? xa + 2 * j : xb + 2 * j - 4;
            x[0] = make_float2(fmaf(x[0].x, cs[j].x, -(x[0].y * sn[j].x)), fmaf(x[0].y, cs[j].x, x[0].x * sn[j].x));
            x[1] = make_float2(fmaf(x[1].x, cs[j].y, -(x[1].y * sn[j].y)), fmaf(x[1].y, cs[j].y, x[1].x * sn[j].y));
          } else {
            const float2 ys = dev::mul2(xb[j], sn[j]), xs = dev::mul2(xa[j], sn[j]);
            xa[j] = make_float2(fmaf(xa[j].x, cs[j].x, -ys.x), fmaf(xa[j].y, cs[j].y, -ys.y));
            xb[j] = dev::fma2(xb[j], cs[j], xs);
          }
        }
      }
      a = to_halves(xa);
      b = to_halves(xb);
    }
    if (q) {
      if (in) {
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + (cur.t * p.num_q_heads + h) * D);
        dst[c0] = a;
        dst[c1] = b;
      }
    } else {
      const bool valid = slot >= 0 && slot < p.num_slots, put = in && valid;
      if (lane == 0 && cur.s == steps.q && slot != -1 && !valid) dev::set_error(p.err, PKV_DEVERR_SLOT_RANGE);
      const int64_t rec = valid ? (slot >> 4) * p.num_kv_heads + h : 0;  // the head's block
      const int r = (int)(slot & 15);
      if constexpr (KV == PKV_KV_INT4) {
        uint32_t* amax = reinterpret_cast<uint32_t*>(chunk_amax) + 2 * (threadIdx.x - pc);  // this head's chunks
        amax[c0] = dev::f16x8_amax_bits(a);
        amax[c1] = dev::f16x8_amax_bits(b);
        __syncwarp();
        const uint4 m0 = reinterpret_cast<const uint4*>(amax)[c0 >> 2], m1 = reinterpret_cast<const uint4*>(amax)[c1 >> 2];
        __syncwarp();  // read before the next step's go over them
        if (put) {
          using R = Int4Record<D>;
          const __half s0 = dev::int4_scale(max(max(m0.x, m0.y), max(m0.z, m0.w)));
          const __half s1 = dev::int4_scale(max(max(m1.x, m1.y), max(m1.z, m1.w)));
          unsigned char* dst = p.cache_k + rec * R::BYTES;
          *reinterpret_cast<uint32_t*>(dst + R::code_at(v, r, c0)) = dev::int4_encode8(a, s0);
          *reinterpret_cast<uint32_t*>(dst + R::code_at(v, r, c1)) = dev::int4_encode8(b, s1);
          if ((c0 & 3) == 0) *reinterpret_cast<__half*>(dst + R::scale_at(v, r, c0)) = s0;
          if ((c1 & 3) == 0) *reinterpret_cast<__half*>(dst + R::scale_at(v, r, c1)) = s1;
        }
      } else if constexpr (KV == PKV_KV_E4M3) {
        const uint32_t m = dev::row_amax_bits<PC>(max(dev::f16x8_amax_bits(a), dev::f16x8_amax_bits(b)));
        if (put) {
          const int sb = dev::e4m3_scale_byte(m);
          uint2* dst = reinterpret_cast<uint2*>((v ? p.cache_v : p.cache_k) + (rec * 16 + r) * D);
          dst[c0] = dev::e4m3_encode8(a, sb);
          dst[c1] = dev::e4m3_encode8(b, sb);
          if (pc == 0) p.scales[rec * 32 + (v ? 16 : 0) + r] = (unsigned char)sb;
        }
      } else if (put) {
        uint4* dst = reinterpret_cast<uint4*>((v ? p.cache_v : p.cache_k) + (rec * 16 + r) * (2 * D));
        dst[c0] = a;
        dst[c1] = b;
      }
    }
    if (cur.s + 1 == steps.all()) {
      fresh = true;
      slot = next_slot;
      pos = next_pos;
    }
    advance(cur);
  };
  for (int i = 0; i < count; i += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u > 0 && i + u >= count) break;
      process(a[u], b[u]);
      load(ahead, i + u + 2 < count, a[u], b[u]);
      advance(ahead);
    }
  }
}

__global__ void __launch_bounds__(256) positions_kernel(const int32_t* __restrict__ context_lens,
                                                        const int32_t* __restrict__ qsl, int num_seqs, int num_tokens,
                                                        int32_t* __restrict__ positions, int32_t* err) {
  dev::griddep_wait();
  dev::griddep_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < num_tokens; i += (int64_t)gridDim.x * blockDim.x) {
    const int t = (int)i, b = dev::row_of_token(qsl, num_seqs, t);
    const int q0 = __ldg(qsl + b), q1 = __ldg(qsl + b + 1), ctx = __ldg(context_lens + b);
    const bool ok = t >= q0 && t < q1 && ctx >= q1 - q0;
    if (!ok) dev::set_error(err, PKV_DEVERR_ROW_META);
    positions[t] = ok ? ctx - (q1 - q0) + (t - q0) : 0;
  }
}

template <int D>
cudaError_t launch_rope(const RopeParams& p, const RopeTurns& turns, int kv_dtype, bool inter, cudaStream_t s) {
  const dim3 grid((unsigned)((p.num_tokens + p.tokens - 1) / p.tokens)), block(kThreads);
  auto* kernel = kv_dtype == PKV_KV_INT4 ? (inter ? rope_append_kernel<D, PKV_KV_INT4, true> : rope_append_kernel<D, PKV_KV_INT4, false>)
                 : kv_dtype == PKV_KV_E4M3
                     ? (inter ? rope_append_kernel<D, PKV_KV_E4M3, true> : rope_append_kernel<D, PKV_KV_E4M3, false>)
                     : (inter ? rope_append_kernel<D, PKV_KV_F16, true> : rope_append_kernel<D, PKV_KV_F16, false>);
  return launch_pdl(kernel, grid, block, 0, s, p, turns);
}

template <int D>
cudaError_t launch_norm(const RopeParams& p, const RopeTurns& turns, int kv_dtype, bool inter, int num_sms, cudaStream_t s) {
  const int64_t steps = (int64_t)p.num_tokens * NormSteps<D>(p.num_q_heads, p.num_kv_heads).all();
  const dim3 grid((unsigned)std::min<int64_t>((steps + kThreads / 32 - 1) / (kThreads / 32), (int64_t)num_sms * kNormCtas)), block(kThreads);
  auto* kernel =
      kv_dtype == PKV_KV_INT4 ? (inter ? norm_rope_append_kernel<D, PKV_KV_INT4, true> : norm_rope_append_kernel<D, PKV_KV_INT4, false>)
      : kv_dtype == PKV_KV_E4M3
          ? (inter ? norm_rope_append_kernel<D, PKV_KV_E4M3, true> : norm_rope_append_kernel<D, PKV_KV_E4M3, false>)
          : (inter ? norm_rope_append_kernel<D, PKV_KV_F16, true> : norm_rope_append_kernel<D, PKV_KV_F16, false>);
  return launch_pdl(kernel, grid, block, 0, s, p, turns);
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_rope_create(const pkv_rope_config* cfg, pkv_rope** out) {
  clear_error();
  if (!cfg || !out) return fail(PKV_ERR_INVALID_ARG, "cfg and out must be non-NULL");
  pkv_rope_config c = *cfg;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (c.rot_dim == 0) c.rot_dim = c.head_dim;
  if (c.rot_dim < 0 || c.rot_dim > c.head_dim) return fail(PKV_ERR_INVALID_ARG, "rot_dim must be in [0, head_dim]");
  if (c.rot_dim % 16 != 0) return fail(PKV_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (c.layout != PKV_ROPE_HALF && c.layout != PKV_ROPE_INTERLEAVED) return fail(PKV_ERR_INVALID_ARG, "unknown layout");
  if (c.scaling < PKV_ROPE_SCALE_NONE || c.scaling > PKV_ROPE_SCALE_RAMP) return fail(PKV_ERR_INVALID_ARG, "unknown scaling");
  if (!(c.base > 1.0) || !std::isfinite(c.base)) return fail(PKV_ERR_INVALID_ARG, "base must be above 1");
  if (c.output_scale == 0.0) c.output_scale = 1.0;
  if (!std::isfinite((float)c.output_scale)) return fail(PKV_ERR_INVALID_ARG, "output_scale must be finite in 32 bits");
  if (c.scaling != PKV_ROPE_SCALE_NONE && (!(c.factor > 0.0) || !std::isfinite(c.factor)))
    return fail(PKV_ERR_INVALID_ARG, "factor must be positive");
  if (c.scaling == PKV_ROPE_SCALE_BANDS || c.scaling == PKV_ROPE_SCALE_RAMP) {
    if (!(c.original_context > 0.0) || !std::isfinite(c.original_context))
      return fail(PKV_ERR_INVALID_ARG, "original_context must be positive");
    if (c.low_turns == 0.0 && c.high_turns == 0.0) {
      c.low_turns = 1.0;
      c.high_turns = c.scaling == PKV_ROPE_SCALE_BANDS ? 4.0 : 32.0;
    }
    if (!(c.low_turns > 0.0) || !(c.high_turns > c.low_turns) || !std::isfinite(c.high_turns))
      return fail(PKV_ERR_INVALID_ARG, "turns must satisfy 0 < low_turns < high_turns");
  }
  pkv_rope* r = new (std::nothrow) pkv_rope();
  if (!r) return fail(PKV_ERR_INVALID_ARG, "out of host memory");
  r->cfg = c;
  auto pair_of = [&](double turns) {
    return c.rot_dim * std::log(c.original_context / (kTwoPi * turns)) / (2.0 * std::log(c.base));
  };
  double lo = 0.0, hi = 0.0;
  if (c.scaling == PKV_ROPE_SCALE_RAMP) {
    lo = std::max(std::floor(pair_of(c.high_turns)), 0.0);
    hi = std::min(std::ceil(pair_of(c.low_turns)), (double)(c.rot_dim - 1));
  }
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = std::pow(c.base, -2.0 * i / c.rot_dim), w = 1.0;
    switch (c.scaling) {
      case PKV_ROPE_SCALE_LINEAR: w = 0.0; break;
      case PKV_ROPE_SCALE_BANDS:
        w = std::min(1.0, std::max(0.0, (c.original_context * f / kTwoPi - c.low_turns) / (c.high_turns - c.low_turns)));
        break;
      case PKV_ROPE_SCALE_RAMP: w = 1.0 - std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001))); break;
      default: break;
    }
    if (w < 1.0) f = w * f + (1.0 - w) * f / c.factor;
    if (!std::isfinite(f)) {
      delete r;
      return fail(PKV_ERR_INVALID_ARG, "factor is too small: a frequency is not finite");
    }
    r->freq[i] = f;
    const double turn = f / kTwoPi;  // whole turns drop out (a factor below 1 can make it pass one)
    r->turn[i] = (uint64_t)std::ldexp(turn - std::floor(turn), 64);
  }
  *out = r;
  return PKV_OK;
}

extern "C" void pkv_rope_destroy(pkv_rope* rope) { delete rope; }

extern "C" int32_t pkv_rope_frequencies(const pkv_rope* rope, double* out, int32_t n) {
  if (!rope) return 0;
  const int32_t cnt = rope->cfg.rot_dim / 2;
  if (out)
    for (int32_t i = 0; i < n && i < cnt; ++i) out[i] = rope->freq[i];
  return cnt;
}

extern "C" pkv_status pkv_positions(pkv_pool* pool, const int32_t* context_lens, const int32_t* query_start_loc,
                                    int32_t num_seqs, int32_t num_tokens, int32_t* positions, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (num_tokens < 0 || num_seqs < 0) return fail(PKV_ERR_INVALID_ARG, "sizes must be >= 0");
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs < 1) return fail(PKV_ERR_INVALID_ARG, "tokens without rows");
  if (!context_lens || !query_start_loc || !positions)
    return fail(PKV_ERR_INVALID_ARG, "metadata pointers must be non-NULL");
  pkv_status st = check_device(pool);
  if (st == PKV_OK) st = validate_metadata(pool, nullptr, 1 << 27, context_lens, query_start_loc, num_seqs, num_tokens, nullptr,
                                           stream);
  if (st != PKV_OK) return st;
  const int blocks = (int)std::min<int64_t>(((int64_t)num_tokens + 255) / 256, pool->num_sms * 8);
  const cudaError_t e = launch_pdl(positions_kernel, dim3(blocks), dim3(256), 0, (cudaStream_t)stream, context_lens,
                                   query_start_loc, (int)num_seqs, (int)num_tokens, positions, pool->dev_error);
  if (e != cudaSuccess) return cuda_fail(e, "positions launch");
  pool->last_launches = 1;
  return PKV_OK;
}

// The norms of a call: null weights leave the heads as they are.
struct HeadNorms {
  const void* q_weight = nullptr;
  const void* k_weight = nullptr;
  float eps = 0.f, offset = 0.f;
};

// Rotation (none with a null rope) and append, with norms in front where `norms` is given.
static pkv_status rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const HeadNorms* norms, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens, void* q_out,
                              void* stream) {
  const pkv_config& c = pool->cfg;
  if (rope && rope->cfg.head_dim != c.head_dim) return fail(PKV_ERR_INVALID_ARG, "rope and pool differ in head_dim");
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens must be >= 0");
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || (rope && !positions) || !slot_mapping)
    return fail(PKV_ERR_INVALID_ARG, "k, v, positions and slot_mapping must be non-NULL");
  if ((q == nullptr) != (q_out == nullptr)) return fail(PKV_ERR_INVALID_ARG, "q and q_out go together");
  const uintptr_t all = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                        reinterpret_cast<uintptr_t>(q_out);
  if (all % 16 != 0) return fail(PKV_ERR_INVALID_ARG, "q, k, v and q_out must be 16-byte aligned");
  const int64_t qw = (int64_t)c.num_q_heads * c.head_dim, kw = (int64_t)c.num_kv_heads * c.head_dim;
  if ((q && (q_stride < qw || q_stride % 8 != 0)) || k_stride < kw || k_stride % 8 != 0 || v_stride < kw || v_stride % 8 != 0)
    return fail(PKV_ERR_INVALID_ARG, "strides must be multiples of 8 and hold a token's heads");
  if (q && q == q_out && q_stride != qw) return fail(PKV_ERR_INVALID_ARG, "q_out may be q only when q is packed");
  pkv_status st = check_device(pool);
  if (st == PKV_OK) st = validate_metadata(pool, nullptr, 0, nullptr, nullptr, 0, num_tokens, slot_mapping, stream);
  if (st != PKV_OK) return st;
  RopeParams p;
  p.q = static_cast<const __half*>(q);
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.q_out = static_cast<__half*>(q_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slot_mapping;
  p.cache_k = static_cast<unsigned char*>(pkv_pool_layer_ptr(pool, layer, 0));
  p.cache_v = static_cast<unsigned char*>(pkv_pool_layer_ptr(pool, layer, 1));
  p.scales = static_cast<unsigned char*>(pkv_pool_scales_ptr(pool, layer));
  p.num_slots = (int64_t)c.num_blocks * c.block_size;
  p.num_tokens = num_tokens;
  p.num_q_heads = q ? c.num_q_heads : 0;
  p.num_kv_heads = c.num_kv_heads;
  p.rot_dim = rope ? rope->cfg.rot_dim : 0;
  p.out_scale = rope ? (float)rope->cfg.output_scale : 1.f;
  p.err = pool->dev_error;
  const HeadNorms none;
  const HeadNorms& hn = norms ? *norms : none;
  p.q_weight = q ? static_cast<const __half*>(hn.q_weight) : nullptr;
  p.k_weight = static_cast<const __half*>(hn.k_weight);
  p.eps = hn.eps;
  p.weight_offset = hn.offset;
  // Two items a thread, in up to four tokens a CTA (larger CTAs start and end in coarser steps: 256 threads and twice
  // the items took 13.3 us where these take 12.4, 8192 tokens of 12 / 2 heads at d 128); fewer while that would leave
  // SMs without two CTAs.
  const int64_t per = (int64_t)(p.num_q_heads + p.num_kv_heads) * (c.head_dim / 16);
  const int64_t fill = std::max<int64_t>(1, 2 * 128 / per), spread = std::max<int64_t>(1, num_tokens / (2 * (int64_t)pool->num_sms));
  p.tokens = (int)std::min<int64_t>(4, std::min(fill, spread));
  RopeTurns turns = {};
  if (rope) std::copy(rope->turn, rope->turn + kMaxPairs, turns.turn);
  const bool inter = rope && rope->cfg.layout == PKV_ROPE_INTERLEAVED;
  const int kv = c.kv_dtype;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e =
      norms ? (c.head_dim == 64    ? launch_norm<64>(p, turns, kv, inter, pool->num_sms, s)
               : c.head_dim == 128 ? launch_norm<128>(p, turns, kv, inter, pool->num_sms, s)
                                   : launch_norm<256>(p, turns, kv, inter, pool->num_sms, s))
            : (c.head_dim == 64    ? launch_rope<64>(p, turns, kv, inter, s)
               : c.head_dim == 128 ? launch_rope<128>(p, turns, kv, inter, s)
                                   : launch_rope<256>(p, turns, kv, inter, s));
  if (e != cudaSuccess) return cuda_fail(e, "rope_append launch");
  note_append(pool, layer);
  pool->last_launches = 1;
  return PKV_OK;
}

extern "C" pkv_status pkv_rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens,
                                      void* q_out, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (layer < 0 || layer >= pool->cfg.num_layers) return fail(PKV_ERR_OUT_OF_RANGE, "layer out of range");
  if (!rope) return fail(PKV_ERR_INVALID_ARG, "rope is NULL");
  return rope_append(pool, layer, rope, nullptr, q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, num_tokens,
                     q_out, stream);
}

extern "C" pkv_status pkv_norm_rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const void* q_weight,
                                           const void* k_weight, float eps, float weight_offset, const void* q, int64_t q_stride,
                                           const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                           const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens,
                                           void* q_out, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (layer < 0 || layer >= pool->cfg.num_layers) return fail(PKV_ERR_OUT_OF_RANGE, "layer out of range");
  if (!q_weight && !k_weight) return fail(PKV_ERR_INVALID_ARG, "no weights: pkv_rope_append is the call without norms");
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) % 16 != 0)
    return fail(PKV_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  if (!(eps >= 1e-30f) || !std::isfinite(eps)) return fail(PKV_ERR_INVALID_ARG, "eps must be finite and at least 1e-30");
  // (times the root's reciprocal, up to 1e15, it stays finite: a head of zeros stays zeros)
  if (!(std::fabs(weight_offset) <= 1e20f)) return fail(PKV_ERR_INVALID_ARG, "weight_offset must be at most 1e20 in magnitude");
  const HeadNorms norms{q_weight, k_weight, eps, weight_offset};
  return rope_append(pool, layer, rope, &norms, q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, num_tokens, q_out,
                     stream);
}
