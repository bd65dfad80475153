// Rotary positions, fused with the append.
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
// Bound by memory: q, k and v read once, q_out and the slots written once.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

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
// A thread loads its first items before it computes its angles, so that neither waits for the other.
template <int D, bool F8, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p, const __grid_constant__ RopeTurns turns) {
  constexpr int PC = D / 16;  // items per head: a power of two within a warp
  constexpr int U = 2;        // items in flight a thread
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
      if constexpr (F8) {
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
cudaError_t launch_rope(const RopeParams& p, const RopeTurns& turns, bool f8, bool inter, cudaStream_t s) {
  const dim3 grid((unsigned)((p.num_tokens + p.tokens - 1) / p.tokens)), block(kThreads);
  if (f8) return inter ? launch_pdl(rope_append_kernel<D, true, true>, grid, block, 0, s, p, turns)
                       : launch_pdl(rope_append_kernel<D, true, false>, grid, block, 0, s, p, turns);
  return inter ? launch_pdl(rope_append_kernel<D, false, true>, grid, block, 0, s, p, turns)
               : launch_pdl(rope_append_kernel<D, false, false>, grid, block, 0, s, p, turns);
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

extern "C" pkv_status pkv_rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens,
                                      void* q_out, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (layer < 0 || layer >= pool->cfg.num_layers) return fail(PKV_ERR_OUT_OF_RANGE, "layer out of range");
  if (!rope) return fail(PKV_ERR_INVALID_ARG, "rope is NULL");
  const pkv_config& c = pool->cfg;
  if (rope->cfg.head_dim != c.head_dim) return fail(PKV_ERR_INVALID_ARG, "rope and pool differ in head_dim");
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens must be >= 0");
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !positions || !slot_mapping)
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
  p.rot_dim = rope->cfg.rot_dim;
  p.out_scale = (float)rope->cfg.output_scale;
  p.err = pool->dev_error;
  // Two items a thread, in up to four tokens a CTA (larger CTAs start and end in coarser steps: 256 threads and twice
  // the items took 13.3 us where these take 12.4, 8192 tokens of 12 / 2 heads at d 128); fewer while that would leave
  // SMs without two CTAs.
  const int64_t per = (int64_t)(p.num_q_heads + p.num_kv_heads) * (c.head_dim / 16);
  const int64_t fill = std::max<int64_t>(1, 2 * 128 / per), spread = std::max<int64_t>(1, num_tokens / (2 * (int64_t)pool->num_sms));
  p.tokens = (int)std::min<int64_t>(4, std::min(fill, spread));
  RopeTurns turns;
  std::copy(rope->turn, rope->turn + kMaxPairs, turns.turn);
  const bool f8 = c.kv_dtype == PKV_KV_E4M3, inter = rope->cfg.layout == PKV_ROPE_INTERLEAVED;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = c.head_dim == 64    ? launch_rope<64>(p, turns, f8, inter, s)
                        : c.head_dim == 128 ? launch_rope<128>(p, turns, f8, inter, s)
                                            : launch_rope<256>(p, turns, f8, inter, s);
  if (e != cudaSuccess) return cuda_fail(e, "rope_append launch");
  note_append(pool, layer);
  pool->last_launches = 1;
  return PKV_OK;
}
