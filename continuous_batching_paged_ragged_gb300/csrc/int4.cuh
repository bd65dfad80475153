// The 4-bit cache's rows: layout of a record, and the conversions both ways.
//
// A (block, KV head) is one record of 18 head_dim bytes:
//     K's codes [head_dim / 32][16 tokens][16 bytes], V's codes likewise, scales [16 tokens][K, V][head_dim / 32] fp16.
// 32 consecutive values of a row share a scale s; byte i of their 16 holds values 2i (lower half) and 2i + 1, each as its
// code plus 8.  Every 16-byte piece of a row lies beside its neighbours' pieces, so that the eight rows which one
// ldmatrix takes are 128 consecutive bytes (no swizzle, no bank conflicts) and a record is one bulk copy.
//
// A code stands for code * s, which is an fp16 number: |code| <= 7 has three bits and s at most eight.  s is the smallest
// number of at most eight significant bits (and a multiple of 2^-24) that is no less than a seventh of the group's largest
// magnitude, but at most 9344, seven of which are 65408: beyond that (65440, 65472 and 65504, which have a seventh up to 9357.7,
// and codes of 7 all the same) the next scale's 7 would pass the fp16 maximum.  A code is the integer nearest to x / s, ties to
// even; nothing is clipped.  What this costs against a scale of 11 bits is a step wider by at most 2^-7; what it gives is that
// every reader of the cache computes with the same values, exactly.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "pkv_internal.cuh"

namespace pkv {

constexpr int kI4Group = 32;  // values that share a scale

template <int D>
struct Int4Record {
  static constexpr int GROUPS = D / kI4Group;
  static constexpr int VALUES = 8 * D;       // offset of V's codes (K's are at 0); bytes of either
  static constexpr int SCALES = 16 * D;      // offset of the scales
  static constexpr int SCALE_ROW = D / 8;    // bytes of a token's scales: K's D / 16, then V's
  static constexpr int BYTES = 18 * D;
  // Chunk c (8 values: 4 bytes of codes) of token r, K (kv = 0) or V, and the scale of its group.
  __host__ __device__ static constexpr int code_at(int kv, int r, int c) { return kv * VALUES + (c >> 2) * 256 + r * 16 + (c & 3) * 4; }
  __host__ __device__ static constexpr int scale_at(int kv, int r, int c) { return SCALES + r * SCALE_ROW + (kv * GROUPS + (c >> 2)) * 2; }
};
// Bytes of a record for any head_dim.
__host__ __device__ constexpr int int4_record_bytes(int head_dim) { return 18 * head_dim; }

namespace dev {

// The scale of a group whose largest magnitude has fp16 bits `amax`.  A seventh is taken a little low (by 2^-20, more than
// the product's rounding) and rounded up to eight significant bits: amax / 7 is either a number of eight bits or off any
// such number by more than 2^-13 of it (amax has 11 bits, seven times eight bits have 11 as well), so the result is the one
// that the exact quotient gives.  Finite magnitudes past 65408 give 9408, which becomes 9344 (infinities and NaN stay what they
// are, and show).  Then up to a multiple of 2^-24, which concerns scales below 2^-16 alone.
__device__ __forceinline__ __half int4_scale(uint32_t amax) {
  const float seventh = __half2float(__ushort_as_half((unsigned short)amax)) * (1.f / 7.f * (1.f - 0x1p-20f));
  const uint32_t b = (__float_as_uint(seventh) + 0xFFFFu) & 0xFFFF0000u;
  return __float2half_ru(b == __float_as_uint(9408.f) ? 9344.f : __uint_as_float(b));
}

// Codes of 8 fp16 values under scale s, value i in bits 4i .. 4i + 3, plus 8.  x / s is x times a rounded reciprocal, off by
// less than 2^-20 for quotients up to 7.02; rounding it to a multiple of 2^-14 first lands on every tie exactly, because a
// quotient that is no tie is at least 2^-12 away from one (x has 11 bits, s eight).  Then to the nearest integer, ties to
// even, in the low bits of a float of ulp 1.
__device__ __forceinline__ uint32_t int4_encode8(const uint4& r, __half s) {
  const float sf = __half2float(s), inv = sf > 0.f ? 1.f / sf : 0.f;
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    c[2 * i] = __float_as_uint(__fadd_rn(__fadd_rn(__fmaf_rn(f.x, inv, 768.f), -768.f), 12582920.f));
    c[2 * i + 1] = __float_as_uint(__fadd_rn(__fadd_rn(__fmaf_rn(f.y, inv, 768.f), -768.f), 12582920.f));
  }
  uint32_t out = c[0] & 15u;
#pragma unroll
  for (int i = 1; i < 8; ++i) out |= (c[i] & 15u) << (4 * i);
  return out;
}

// Eight codes as fp16 values code * s, exactly.
__device__ __forceinline__ uint4 int4x8_dequant(uint32_t codes, __half s) {
  const __half2 s2 = __half2half2(s);
  uint32_t p[4];  // pairs (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((codes >> (4 * i)) & 0x000F000Fu) | 0x64006400u;  // 1024 + code + 8
    __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half(0x6408)));
    v = __hmul2(v, s2);
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                    __byte_perm(p[2], p[3], 0x7632));
}

// The largest magnitude over a group's four lanes (lane-aligned; every lane of the warp takes part).
__device__ __forceinline__ uint32_t int4_group_amax(const uint4& r) { return row_amax_bits<4>(f16x8_amax_bits(r)); }

}  // namespace dev
}  // namespace pkv
