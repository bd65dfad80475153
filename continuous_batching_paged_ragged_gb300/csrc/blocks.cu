// Copying, forking and compacting blocks of the cache, every layer at once.
//
// "Continuous Batching Is Not a Bigger Batch", section "The allocator is the other half": requests hold blocks and
// a freed block becomes another request's.  What a block holds is spread over the pool: in each of the
// 2 * num_layers planes [num_blocks][Hkv][16][d] (K and V of a layer) one contiguous piece of Hkv * 16 * d values,
// and on an 8-bit cache in each of num_layers scale planes one piece of Hkv 32-byte records.  On a 4-bit cache it is Hkv
// whole records in each of num_layers planes (int4.cuh).  Nothing is computed: the calls are bound by memory, every moved
// byte read once and written once.
#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "int4.cuh"
#include "pkv_internal.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kForkCtas = 6;  // fork_rows: CTAs per SM (copy_rows)
constexpr int kBS = 16;

struct BlockGeo {
  char* values;            // [planes][num_blocks][num_kv_heads][16][row_bytes]
  unsigned char* scales;   // 8-bit: [num_layers][num_blocks][num_kv_heads][2][16] bytes, else null
  int64_t plane_bytes;     // of a value plane
  int64_t scale_bytes;     // of a scale plane
  int planes;              // value planes: 2 * num_layers (4-bit: num_layers, of records)
  int scale_planes;        // num_layers, or 0
  int num_kv_heads, row_bytes, num_blocks;  // row_bytes: a sixteenth of a (block, head)'s piece
  int32_t* err;
};

BlockGeo geo_of(const pkv_pool* pool) {
  const pkv_config& c = pool->cfg;
  const bool f8 = c.kv_dtype == PKV_KV_E4M3;
  BlockGeo g;
  g.values = pool->base;
  g.scales = f8 ? reinterpret_cast<unsigned char*>(pool->base + pool->scales_off) : nullptr;
  const bool i4 = c.kv_dtype == PKV_KV_INT4;
  g.row_bytes = i4 ? int4_record_bytes(c.head_dim) / kBS : c.head_dim * (f8 ? 1 : 2);
  g.plane_bytes = (int64_t)c.num_blocks * c.num_kv_heads * kBS * g.row_bytes;
  g.scale_bytes = (int64_t)c.num_blocks * c.num_kv_heads * 32;
  g.planes = (i4 ? 1 : 2) * c.num_layers;
  g.scale_planes = f8 ? c.num_layers : 0;
  g.num_kv_heads = c.num_kv_heads;
  g.num_blocks = c.num_blocks;
  g.err = pool->dev_error;
  return g;
}

// The first `rows` rows of every head of block src into block dst, planes [p0, p1) of the planes + scale_planes,
// by all threads of the CTA.  A warp takes the pieces (plane, head) in turn, kPieces at once so that its lanes have
// loads in flight however short a piece is (one row is 64 bytes or more, all sixteen 1 to 8 KB); nothing is divided in
// the loop.  Forks are bound by this loop's instructions and latency, not by DRAM (a parent's children share its reads
// through L2, and the writes stay there): 288 forks over 28 layers of an 8-bit cache take 14.2 us (4.7 TB/s read and
// written) with four pieces and six CTAs an SM, 16 with two and eight, 18 with a divided index for every chunk.
__device__ void copy_rows(const BlockGeo& g, int src, int dst, int rows, int p0, int p1) {
  constexpr int kPieces = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = kBS * g.row_bytes / 16;    // 16-byte chunks of a head's run
  const int live = rows * g.row_bytes / 16;  // of which copied
  const int64_t plane = g.plane_bytes / 16;
  const int v1 = min(p1, g.planes), n = max(0, v1 - p0) * g.num_kv_heads;
  const uint4* in = reinterpret_cast<const uint4*>(g.values) + (int64_t)src * g.num_kv_heads * run + p0 * plane;
  uint4* out = reinterpret_cast<uint4*>(g.values) + (int64_t)dst * g.num_kv_heads * run + p0 * plane;
  for (int i0 = warp * kPieces; i0 < n; i0 += kThreads / 32 * kPieces) {
    int64_t off[kPieces];
    int p = i0 / g.num_kv_heads, h = i0 - p * g.num_kv_heads;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      off[k] = p * plane + h * run;
      if (++h == g.num_kv_heads) {
        h = 0;
        ++p;
      }
    }
    for (int c = lane; c < live; c += 32) {
      uint4 v[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        if (i0 + k < n) v[k] = __ldcs(in + off[k] + c);
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        if (i0 + k < n) __stcs(out + off[k] + c, v[k]);
    }
  }
  // 8-bit: one thread a scale record (16 slots of K or V of a head), the first `rows` bytes of it
  const int s0 = max(p0, g.planes) - g.planes, s1 = p1 - g.planes;
  const int recs = 2 * g.num_kv_heads;
  for (int i = threadIdx.x; i < (s1 - s0) * recs; i += kThreads) {
    const int p = s0 + i / recs, r = i % recs;
    const int64_t off = p * g.scale_bytes + (int64_t)r * 16;
    const uint4 v = *reinterpret_cast<const uint4*>(g.scales + off + (int64_t)src * recs * 16);
    unsigned char* to = g.scales + off + (int64_t)dst * recs * 16;
    if (rows & 8) *reinterpret_cast<uint2*>(to) = make_uint2(v.x, v.y);
    const uint32_t four = rows & 8 ? v.z : v.x, rest = rows & 8 ? (rows & 4 ? v.w : v.z) : (rows & 4 ? v.y : v.x);
    if (rows & 4) *reinterpret_cast<uint32_t*>(to + (rows & 8)) = four;
    if (rows & 2) *reinterpret_cast<uint16_t*>(to + (rows & 12)) = (uint16_t)rest;
    if (rows & 1) to[rows & 14] = (unsigned char)(rest >> (rows & 2 ? 16 : 0));
  }
}

// The same on a 4-bit cache: of every record the first `rows` of the 16 pieces of each group's codes, and the scales' first
// `rows` rows (8 bytes or more each).  A warp takes a record at a time.  288 forks with tails of nine tokens over 28 layers of two
// heads at d 128: 11.7 us for a floor of 3.5 (8-bit 13.6 for 6.3, fp16 20.0 for 12.5), as the forks above instructions and latency.
__device__ void copy_rows_int4(const BlockGeo& g, int src, int dst, int rows, int p0, int p1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int record = kBS * g.row_bytes, head_dim = record / 18;
  const int chunks = head_dim;                    // 16-byte pieces of K's and V's codes: 2 * (head_dim / 32) * 16
  const int words = rows * (head_dim / 64);       // 8-byte words of the scales
  const int n = (p1 - p0) * g.num_kv_heads;
  for (int i = warp; i < n; i += kThreads / 32) {
    const int p = p0 + i / g.num_kv_heads, h = i % g.num_kv_heads;
    const char* in = g.values + p * g.plane_bytes + ((int64_t)src * g.num_kv_heads + h) * record;
    char* out = g.values + p * g.plane_bytes + ((int64_t)dst * g.num_kv_heads + h) * record;
    constexpr int U = 4;  // loads in flight a lane
    for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < chunks && (c0 & 15) < rows) v[u] = __ldcs(reinterpret_cast<const uint4*>(in) + c0 + 32 * u);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < chunks && (c0 & 15) < rows) __stcs(reinterpret_cast<uint4*>(out) + c0 + 32 * u, v[u]);
    }
    for (int c = lane; c < words; c += 32)
      reinterpret_cast<uint2*>(out + 16 * head_dim)[c] = reinterpret_cast<const uint2*>(in + 16 * head_dim)[c];
  }
}

// End of a kernel that writes cached rows.  The attention kernels stream their first blocks before their dependency
// wait (only appends release their dependents earlier, and the attention call knows of those: append_since).  So the
// kernels below release their dependents by ending, every thread's writes performed by then.
__device__ __forceinline__ void publish() {
  __threadfence();
  dev::fence_proxy_async_global();
}

__device__ __forceinline__ bool bad_block(const BlockGeo& g, int id) { return id < 0 || id >= g.num_blocks; }

// The planes of one unit of work: slice s of `slices`.
__device__ __forceinline__ void slice_planes(const BlockGeo& g, int s, int slices, int& p0, int& p1) {
  const int all = g.planes + g.scale_planes;
  p0 = (int)((int64_t)all * s / slices);
  p1 = (int)((int64_t)all * (s + 1) / slices);
}

// ---------------------------------------------------------------------------------------------------
// Whole blocks, by the bulk copy engine.  A worker (one thread of a warp of its own) takes pieces of up to kPiece bytes
// of one plane of one move, every worker its own sequence over all moves and planes, through a ring of kSlots buffers
// in shared memory: the load of a piece is issued kSlots - 1 pieces ahead of its store, and nothing passes through
// registers.  Six workers an SM with two pieces each: 1 GB in blocks of 1 MB takes 340 us (6.3 TB/s read and written, 93 % of
// the measured copy rate), 1235 scattered blocks of 458 KB 180 us (93 %).  More in flight does not help (12 workers of
// three 8 KB pieces 340 and 193 us); plain 16-byte loads and stores, which run dry at every unit of work, took 343 and 238.
// ---------------------------------------------------------------------------------------------------
constexpr int kPiece = 16384;
constexpr int kSlots = 2;
constexpr int kWorkers = 3;  // per CTA
constexpr int kBulkSmem = kWorkers * kSlots * kPiece;
constexpr int kBulkCtas = 2;  // per SM

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(dev::smem_addr(src_smem)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the latest N stores have read their buffers.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Where a worker's piece comes from and goes to (bytes 0: nothing to copy).
struct Piece {
  const char* src;
  char* dst;
  uint32_t bytes;
};

// The pieces of a block: every value plane in `parts` parts, then the scale planes whole (in parts of kPiece too).
struct PieceGeo {
  int value_bytes, value_parts;   // of one block in a value plane
  int scale_bytes, scale_parts;
  __device__ explicit PieceGeo(const BlockGeo& g) {
    value_bytes = g.num_kv_heads * kBS * g.row_bytes;
    value_parts = (value_bytes + kPiece - 1) / kPiece;
    scale_bytes = g.num_kv_heads * 32;
    scale_parts = (scale_bytes + kPiece - 1) / kPiece;
  }
  __device__ int per_block(const BlockGeo& g) const { return g.planes * value_parts + g.scale_planes * scale_parts; }
  __device__ Piece piece(const BlockGeo& g, int src, int dst, int q) const {
    const int nv = g.planes * value_parts;
    const bool value = q < nv;
    const int parts = value ? value_parts : scale_parts, block = value ? value_bytes : scale_bytes;
    const int r = value ? q : q - nv, plane = r / parts, at = (r - plane * parts) * kPiece;
    char* base = value ? g.values + plane * g.plane_bytes : reinterpret_cast<char*>(g.scales) + plane * g.scale_bytes;
    return Piece{base + (int64_t)src * block + at, base + (int64_t)dst * block + at, (uint32_t)min(kPiece, block - at)};
  }
};

// Copies `moves` blocks; ends(m, src, dst) gives move m's blocks, or false to skip it.  Called by all threads of a CTA of
// kWorkers warps.
template <typename F>
__device__ void bulk_copy(const BlockGeo& g, int64_t moves, unsigned char* smem, F ends) {
  __shared__ __align__(8) uint64_t full[kWorkers][kSlots];
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) != 0) return;
  for (int s = 0; s < kSlots; ++s) dev::mbar_init(&full[w][s], 1);
  dev::fence_mbar_init();
  dev::fence_proxy_async_smem();
  unsigned char* ring = smem + w * kSlots * kPiece;
  const PieceGeo pg(g);
  const int per = pg.per_block(g);
  const int step = gridDim.x * kWorkers, step_m = step / per, step_q = step % per;
  int64_t m = (blockIdx.x * kWorkers + w) / per;  // the next piece to load: of move m,
  int q = (blockIdx.x * kWorkers + w) % per;      // its piece q
  char* to[kSlots];
  uint32_t bytes[kSlots];
  // the worker's next piece into slot s; none (bytes 0) at the end of its sequence
  auto load = [&](int s) {
    bytes[s] = 0;
    while (m < moves && bytes[s] == 0) {
      int src, dst;
      if (ends(m, q == 0, src, dst)) {
        const Piece p = pg.piece(g, src, dst, q);
        to[s] = p.dst;
        bytes[s] = p.bytes;
        dev::mbar_arrive_expect_tx(&full[w][s], p.bytes);
        dev::bulk_g2s_plain(ring + s * kPiece, p.src, p.bytes, &full[w][s]);
      }
      m += step_m;
      q += step_q;
      if (q >= per) {
        q -= per;
        ++m;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kSlots; ++s) load(s);
  bool ok = true;
  for (uint32_t round = 0; ok; ++round) {
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (bytes[s] == 0) {
        ok = false;
        break;
      }
      if (!dev::mbar_wait(&full[w][s], round & 1)) {
        dev::set_error(g.err, PKV_DEVERR_WAIT_TIMEOUT);
        for (int t = 0; t < kSlots; ++t)  // the copies still in flight
          if (t != s && bytes[t]) dev::mbar_wait(&full[w][t], (t > s ? round : round + 1) & 1);
        ok = false;
        break;
      }
      bulk_s2g(to[s], ring + s * kPiece, bytes[s]);
      // refill the slot before this one: its store is the one issued last but one
      const int e = (s + kSlots - 1) % kSlots;
      if (round > 0 || s > 0) {
        bulk_wait_read<1>();
        load(e);
      }
    }
  }
  bulk_wait_all();
}

__global__ void __launch_bounds__(kWorkers * 32) copy_blocks_kernel(const BlockGeo g, const int32_t* __restrict__ pairs,
                                                                    int num_pairs) {
  extern __shared__ __align__(128) unsigned char smem[];
  dev::griddep_wait();
  bulk_copy(g, num_pairs, smem, [&](int64_t m, bool first, int& src, int& dst) {
    src = __ldg(pairs + 2 * m);
    dst = __ldg(pairs + 2 * m + 1);
    if (src == -1 || dst == -1) return false;
    if (!bad_block(g, src) && !bad_block(g, dst)) return true;
    if (first) dev::set_error(g.err, PKV_DEVERR_BLOCK_RANGE);
    return false;
  });
  publish();
}

template <bool I4>
__global__ void __launch_bounds__(kThreads, kForkCtas) fork_rows_kernel(const BlockGeo g, int32_t* tables, int max_blocks, int32_t* ctx,
                                                             int num_seqs, const int32_t* __restrict__ forks, int num_forks,
                                                             int slices) {
  dev::griddep_wait();
  const int64_t units = (int64_t)num_forks * slices;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t f = u / slices;
    const int s = (int)(u - f * slices);
    const int parent = __ldg(forks + 3 * f), child = __ldg(forks + 3 * f + 1), block = __ldg(forks + 3 * f + 2);
    if (parent == -1) continue;
    const bool first = s == 0 && threadIdx.x == 0;
    if (parent < 0 || parent >= num_seqs || child < 0 || child >= num_seqs || child == parent) {
      if (first) dev::set_error(g.err, PKV_DEVERR_ROW_META);
      continue;
    }
    const int c = ctx[parent];
    if (c < 0 || c > (int64_t)max_blocks * kBS) {
      if (first) dev::set_error(g.err, PKV_DEVERR_ROW_META);
      continue;
    }
    const int full = c / kBS, tail = c % kBS;
    const int32_t* from = tables + (int64_t)parent * max_blocks;
    const int last = tail > 0 ? from[full] : 0;
    if (tail > 0 && (bad_block(g, last) || bad_block(g, block))) {
      if (first) dev::set_error(g.err, PKV_DEVERR_BLOCK_RANGE);
      continue;
    }
    if (s == 0) {
      int32_t* to = tables + (int64_t)child * max_blocks;
      for (int j = threadIdx.x; j < max_blocks; j += blockDim.x) to[j] = j < full ? from[j] : j == full && tail > 0 ? block : -1;
      if (threadIdx.x == 0) ctx[child] = c;
    }
    if (tail > 0) {
      int p0, p1;
      slice_planes(g, s, slices, p0, p1);
      if constexpr (I4) copy_rows_int4(g, last, block, tail, p0, p1); else copy_rows(g, last, block, tail, p0, p1);
    }
  }
  publish();
}

// ---------------------------------------------------------------------------------------------------
// Compaction.  The used blocks as a bitmap; with n of them, the used ids at n and above (ascending) go to the unused
// ids below n (ascending): there are as many of one as of the other, so every block moves at most once and no
// source is a destination.
// ---------------------------------------------------------------------------------------------------
struct CompactHdr {
  int32_t marked;   // marking CTAs that have finished
  int32_t n_moves;
  int32_t pad[62];
};
static_assert(sizeof(CompactHdr) == 256, "one 256-byte line");

struct CompactWs {
  size_t bits, src, dst, total;
};
CompactWs compact_ws(int num_blocks) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  CompactWs w;
  w.bits = sizeof(CompactHdr);
  w.src = w.bits + up(((size_t)num_blocks + 31) / 32 * 4);
  w.dst = w.src + up(((size_t)num_blocks / 2 + 1) * 4);  // at most half of the blocks move
  w.total = w.dst + up(((size_t)num_blocks / 2 + 1) * 4);
  return w;
}

constexpr int kPlanThreads = 1024;
constexpr size_t kPlanBitmap = 47 * 1024;  // bytes of bitmap for one planning CTA: 48 KB, less what its scans share

__device__ int block_scan(int v, int* sums, int* total) {  // exclusive, over kPlanThreads threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int before = warp ? sums[warp - 1] : 0;
  *total = sums[31];
  __syncthreads();  // sums is reused by the next scan
  return before + x - v;
}

struct CompactParams {
  const int32_t* tables;
  int32_t* new_tables;
  int32_t* remap;
  int32_t* num_live;
  CompactHdr* hdr;
  uint32_t* bits;
  int32_t* src;
  int32_t* dst;
  int64_t entries;
  int num_blocks;
  int32_t* err;
};

// Bits of word w of the bitmap's ids below n.
__device__ __forceinline__ uint32_t below(int w, int n) {
  const int64_t k = (int64_t)n - (int64_t)w * 32;
  return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1;
}

// By one CTA of kPlanThreads threads: the moves, remap and the count from the finished bitmap.  Every thread owns a
// run of consecutive words, so that three block-wide scans order all ids.
__device__ void plan_moves(const CompactParams& p, const uint32_t* bits) {
  __shared__ int sums[32];
  const int words = (p.num_blocks + 31) / 32, per = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
  int used = 0;
  for (int w = w0; w < w1; ++w) used += __popc(bits[w]);
  int n = 0, moves = 0, holes = 0;
  block_scan(used, sums, &n);
  int nm = 0, nh = 0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t b = bits[w], lo = below(w, n);
    nm += __popc(b & ~lo);
    nh += __popc(~b & lo);
  }
  int im = block_scan(nm, sums, &moves), ih = block_scan(nh, sums, &holes);
  for (int w = w0; w < w1; ++w) {
    const uint32_t b = bits[w], lo = below(w, n);
    for (uint32_t m = b & ~lo; m; m &= m - 1) p.src[im++] = w * 32 + __ffs(m) - 1;
    for (uint32_t h = ~b & lo; h; h &= h - 1) p.dst[ih++] = w * 32 + __ffs(h) - 1;
  }
  for (int i = threadIdx.x; i < p.num_blocks; i += kPlanThreads) p.remap[i] = bits[i >> 5] >> (i & 31) & 1 ? i : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kPlanThreads) p.remap[p.src[i]] = p.dst[i];
  if (threadIdx.x == 0) {
    p.hdr->n_moves = moves;
    *p.num_live = n;
  }
}

__device__ __forceinline__ void mark(const CompactParams& p, uint32_t* bits, int64_t first, int64_t step) {
  constexpr int U = 4;  // loads in flight a thread
  for (int64_t i0 = first; i0 < p.entries; i0 += U * step) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i0 + u * step < p.entries ? __ldg(p.tables + i0 + u * step) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (id[u] == -1) continue;
      if (id[u] < 0 || id[u] >= p.num_blocks) dev::set_error(p.err, PKV_DEVERR_BLOCK_RANGE);
      else atomicOr(bits + (id[u] >> 5), 1u << (id[u] & 31));
    }
  }
}

// One CTA, the bitmap in its shared memory.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  extern __shared__ uint32_t sbits[];
  dev::griddep_wait();
  dev::griddep_launch_dependents();
  for (int w = threadIdx.x; w < (p.num_blocks + 31) / 32; w += kPlanThreads) sbits[w] = 0;
  __syncthreads();
  mark(p, sbits, threadIdx.x, kPlanThreads);
  __syncthreads();
  plan_moves(p, sbits);
}

// Large tables or pools: the bitmap in the workspace, cleared by a kernel of its own; the last CTA to finish its
// share of the marking plans.
__global__ void __launch_bounds__(kPlanThreads) compact_clear_kernel(const CompactParams p) {
  dev::griddep_wait();
  dev::griddep_launch_dependents();
  const int words = (p.num_blocks + 31) / 32;
  for (int w = blockIdx.x * kPlanThreads + threadIdx.x; w < words; w += gridDim.x * kPlanThreads) p.bits[w] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.hdr->marked = 0;
}

__global__ void __launch_bounds__(kPlanThreads) compact_mark_kernel(const CompactParams p) {
  __shared__ int last;
  dev::griddep_wait();
  dev::griddep_launch_dependents();
  mark(p, p.bits, (int64_t)blockIdx.x * kPlanThreads + threadIdx.x, (int64_t)gridDim.x * kPlanThreads);
  __syncthreads();  // the CTA's marks precede its count
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&p.hdr->marked, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (last) plan_moves(p, p.bits);
}

__global__ void __launch_bounds__(kWorkers * 32) compact_move_kernel(const BlockGeo g, const CompactParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  dev::griddep_wait();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < p.entries; i += (int64_t)gridDim.x * blockDim.x) {
    const int id = p.tables[i];
    p.new_tables[i] = id >= 0 && id < p.num_blocks ? p.remap[id] : id;
  }
  bulk_copy(g, p.hdr->n_moves, smem, [&](int64_t m, bool, int& src, int& dst) {
    src = p.src[m];
    dst = p.dst[m];
    return true;
  });
  publish();
}

// Small pools and tables, in one launch: every CTA makes the whole plan for itself in shared memory (one warp orders the
// ids) and goes on to its pieces; CTA 0 writes the plan out.  The tables are read by every CTA, so they may not be
// rewritten in place here.
constexpr int kSmallEntries = 1024;
constexpr int kSmallBlocks = 2048;

__global__ void __launch_bounds__(kWorkers * 32) compact_small_kernel(const BlockGeo g, const CompactParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t bits[kSmallBlocks / 32];
  __shared__ int32_t src[kSmallBlocks / 2], dst[kSmallBlocks / 2];
  __shared__ int live, moves;
  constexpr int PER = kSmallBlocks / 32 / 32;  // bitmap words a lane
  const int lane = threadIdx.x & 31;
  for (int w = threadIdx.x; w < kSmallBlocks / 32; w += blockDim.x) bits[w] = 0;
  __syncthreads();
  dev::griddep_wait();
  mark(p, bits, threadIdx.x, blockDim.x);
  __syncthreads();
  if (threadIdx.x < 32) {
    auto before = [&](int v, int& total) {  // sum over the lower lanes, and over all
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      total = __shfl_sync(0xffffffffu, x, 31);
      return x - v;
    };
    uint32_t b[PER];
    int used = 0, nm = 0, nh = 0, n, m, h;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      b[k] = bits[lane * PER + k];
      used += __popc(b[k]);
    }
    before(used, n);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const uint32_t lo = below(lane * PER + k, n);
      nm += __popc(b[k] & ~lo);
      nh += __popc(~b[k] & lo);
    }
    int im = before(nm, m), ih = before(nh, h);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int w = lane * PER + k;
      const uint32_t lo = below(w, n);
      for (uint32_t x = b[k] & ~lo; x; x &= x - 1) src[im++] = w * 32 + __ffs(x) - 1;
      for (uint32_t x = ~b[k] & lo; x; x &= x - 1) dst[ih++] = w * 32 + __ffs(x) - 1;
    }
    if (lane == 0) {
      live = n;
      moves = m;
    }
  }
  __syncthreads();
  // a used block's new id: its own below `live`, else that of its move (src ascends)
  auto moved = [&](int id) {
    if (id < live) return id;
    int lo = 0, hi = moves - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (src[mid] <= id) lo = mid; else hi = mid - 1;
    }
    return dst[lo];
  };
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < p.entries; i += (int64_t)gridDim.x * blockDim.x) {
    const int id = __ldg(p.tables + i);
    p.new_tables[i] = id >= 0 && id < p.num_blocks ? moved(id) : id;
  }
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.num_blocks; i += gridDim.x * blockDim.x)
    p.remap[i] = bits[i >> 5] >> (i & 31) & 1 ? moved(i) : -1;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.num_live = live;
  bulk_copy(g, moves, smem, [&](int64_t m, bool, int& s, int& d) {
    s = src[m];
    d = dst[m];
    return true;
  });
  publish();
}

// ---- host -----------------------------------------------------------------------------------------
// Under PKV_VALIDATE=1 (and outside a capture): n int32 of `src` on the host, after the stream's earlier work.
pkv_status fetch_for_validation(const int32_t* src, size_t n, void* stream, std::vector<int32_t>* out, bool* ran) {
  *ran = false;
  const char* env = std::getenv("PKV_VALIDATE");
  if (!env || std::strcmp(env, "1") != 0) return PKV_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &cap);
  if (e != cudaSuccess) return cuda_fail(e, "PKV_VALIDATE: cudaStreamIsCapturing");
  if (cap != cudaStreamCaptureStatusNone) return PKV_OK;
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "PKV_VALIDATE: cudaStreamSynchronize");
  out->resize(n);
  e = cudaMemcpy(out->data(), src, n * 4, cudaMemcpyDefault);
  if (e != cudaSuccess) return cuda_fail(e, "PKV_VALIDATE: copy");
  *ran = true;
  return PKV_OK;
}

// CTAs for up to `moves` block copies: a worker for every piece, up to what is resident at once.
int64_t bulk_grid(const pkv_pool* pool, const BlockGeo& g, int64_t moves) {
  const int64_t pieces = moves * (g.planes + g.scale_planes);  // at least
  return std::max<int64_t>(1, std::min<int64_t>((pieces + kWorkers - 1) / kWorkers, (int64_t)pool->num_sms * kBulkCtas));
}

// Slices of a block's planes for `items` block copies: as many units of work as CTAs are resident at once, or the next
// fewer (a second round would start with the chain of loads that finds a unit's blocks).
int slices_for(const BlockGeo& g, int64_t items, int64_t ctas) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(g.planes + g.scale_planes, ctas / items));
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_copy_blocks(pkv_pool* pool, const int32_t* pairs, int32_t num_pairs, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (num_pairs < 0) return fail(PKV_ERR_INVALID_ARG, "num_pairs must be >= 0");
  if (num_pairs == 0) return PKV_OK;
  if (!pairs) return fail(PKV_ERR_INVALID_ARG, "pairs must be non-NULL");
  pkv_status st = check_device(pool);
  if (st != PKV_OK) return st;
  std::vector<int32_t> host;
  bool ran = false;
  st = fetch_for_validation(pairs, (size_t)num_pairs * 2, stream, &host, &ran);
  if (st != PKV_OK) return st;
  if (ran) {
    std::vector<int> role(pool->cfg.num_blocks, 0);  // 1: a source, 2: a destination
    for (int i = 0; i < num_pairs; ++i) {
      const int32_t s = host[2 * i], d = host[2 * i + 1];
      if (s == -1 || d == -1) continue;
      if (s < 0 || s >= pool->cfg.num_blocks || d < 0 || d >= pool->cfg.num_blocks)
        return fail(PKV_ERR_OUT_OF_RANGE, "PKV_VALIDATE: pair " + std::to_string(i) + " is (" + std::to_string(s) + ", " +
                                              std::to_string(d) + ")");
      if (role[s] == 2 || role[d] != 0 || s == d)
        return fail(PKV_ERR_INVALID_ARG, "PKV_VALIDATE: pair " + std::to_string(i) + ": a destination in another pair");
      role[s] = 1;
      role[d] = 2;
    }
  }
  const BlockGeo g = geo_of(pool);
  cudaError_t e = prepare_kernel(pool, copy_blocks_kernel, kBulkSmem);
  if (e == cudaSuccess)
    e = launch_pdl(copy_blocks_kernel, dim3((unsigned)bulk_grid(pool, g, num_pairs)), dim3(kWorkers * 32), kBulkSmem,
                   (cudaStream_t)stream, g, pairs, (int)num_pairs);
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
  pool->last_launches = 1;
  return PKV_OK;
}

extern "C" pkv_status pkv_fork_rows(pkv_pool* pool, int32_t* block_tables, int32_t max_blocks_per_seq, int32_t* context_lens,
                                    int32_t num_seqs, const int32_t* forks, int32_t num_forks, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (num_forks < 0 || num_seqs < 0) return fail(PKV_ERR_INVALID_ARG, "sizes must be >= 0");
  if (num_forks == 0) return PKV_OK;
  if (max_blocks_per_seq < 1) return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq must be >= 1");
  if (!block_tables || !context_lens || !forks) return fail(PKV_ERR_INVALID_ARG, "metadata pointers must be non-NULL");
  pkv_status st = check_device(pool);
  if (st != PKV_OK) return st;
  std::vector<int32_t> host;
  bool ran = false;
  st = fetch_for_validation(forks, (size_t)num_forks * 3, stream, &host, &ran);
  if (st != PKV_OK) return st;
  if (ran) {
    std::vector<char> child(num_seqs, 0), block(pool->cfg.num_blocks, 0);
    for (int i = 0; i < num_forks; ++i) {
      const int32_t p = host[3 * i], c = host[3 * i + 1], b = host[3 * i + 2];
      if (p == -1) continue;
      if (p < 0 || p >= num_seqs || c < 0 || c >= num_seqs || p == c || child[c])
        return fail(PKV_ERR_INVALID_ARG, "PKV_VALIDATE: fork " + std::to_string(i) + " is of row " + std::to_string(p) +
                                             " into row " + std::to_string(c));
      child[c] = 1;
      if (b >= 0 && b < pool->cfg.num_blocks) {
        if (block[b]) return fail(PKV_ERR_INVALID_ARG, "PKV_VALIDATE: fork " + std::to_string(i) + ": block " +
                                                           std::to_string(b) + " is another fork's");
        block[b] = 1;
      }
    }
    for (int i = 0; i < num_forks; ++i)
      if (host[3 * i] != -1 && child[host[3 * i]])
        return fail(PKV_ERR_INVALID_ARG, "PKV_VALIDATE: row " + std::to_string(host[3 * i]) + " is a child and a parent");
  }
  const BlockGeo g = geo_of(pool);
  const int64_t ctas = (int64_t)pool->num_sms * kForkCtas;
  const int slices = slices_for(g, num_forks, ctas);
  const int64_t grid = std::min<int64_t>((int64_t)num_forks * slices, ctas);
  const cudaError_t e = launch_pdl(pool->cfg.kv_dtype == PKV_KV_INT4 ? fork_rows_kernel<true> : fork_rows_kernel<false>,
                                   dim3((unsigned)grid), dim3(kThreads), 0, (cudaStream_t)stream, g, block_tables,
                                   (int)max_blocks_per_seq, context_lens, (int)num_seqs, forks, (int)num_forks, slices);
  if (e != cudaSuccess) return cuda_fail(e, "fork_rows launch");
  pool->last_launches = 1;
  return PKV_OK;
}

extern "C" size_t pkv_compact_workspace_bytes(const pkv_pool* pool) {
  return pool ? compact_ws(pool->cfg.num_blocks).total : 0;
}

extern "C" pkv_status pkv_compact(pkv_pool* pool, const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t num_seqs,
                                  int32_t* new_tables, int32_t* remap, int32_t* num_live, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  clear_error();
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  pool->last_launches = 0;
  if (num_seqs < 0) return fail(PKV_ERR_INVALID_ARG, "sizes must be >= 0");
  if (max_blocks_per_seq < 1) return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq must be >= 1");
  if (num_seqs > 0 && (!block_tables || !new_tables)) return fail(PKV_ERR_INVALID_ARG, "tables must be non-NULL");
  if (!remap || !num_live || !workspace) return fail(PKV_ERR_INVALID_ARG, "remap, num_live and workspace must be non-NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const int nb = pool->cfg.num_blocks;
  const CompactWs w = compact_ws(nb);
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_INVALID_ARG, "workspace too small: need " + std::to_string(w.total) + " bytes");
  pkv_status st = check_device(pool);
  if (st != PKV_OK) return st;
  char* ws = static_cast<char*>(workspace);
  CompactParams p;
  p.tables = block_tables;
  p.new_tables = new_tables;
  p.remap = remap;
  p.num_live = num_live;
  p.hdr = reinterpret_cast<CompactHdr*>(ws);
  p.bits = reinterpret_cast<uint32_t*>(ws + w.bits);
  p.src = reinterpret_cast<int32_t*>(ws + w.src);
  p.dst = reinterpret_cast<int32_t*>(ws + w.dst);
  p.entries = (int64_t)num_seqs * max_blocks_per_seq;
  p.num_blocks = nb;
  p.err = pool->dev_error;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t smem = ((size_t)nb + 31) / 32 * 4;
  int launches = 0;
  cudaError_t e;
  const BlockGeo g = geo_of(pool);
  const unsigned movers = (unsigned)bulk_grid(pool, g, nb);  // the number of moves is known on the device alone
  const bool apart = p.entries == 0 || new_tables + p.entries <= block_tables || block_tables + p.entries <= new_tables;
  if (p.entries <= kSmallEntries && nb <= kSmallBlocks && apart) {
    e = prepare_kernel(pool, compact_small_kernel, kBulkSmem);
    if (e == cudaSuccess) e = launch_pdl(compact_small_kernel, dim3(movers), dim3(kWorkers * 32), kBulkSmem, s, g, p);
    if (e != cudaSuccess) return cuda_fail(e, "compact launch");
    pool->last_launches = 1;
    return PKV_OK;
  }
  // One CTA marks up to 16 K entries in a few microseconds; past that (or a bitmap that shared memory does not hold) two
  // more launches spread the marking over the GPU.
  if (smem <= kPlanBitmap && p.entries <= 16 * 1024) {
    e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, p);
    launches = 1;
  } else {
    const int64_t clear = std::min<int64_t>((smem / 4 + kPlanThreads - 1) / kPlanThreads, pool->num_sms);
    e = launch_pdl(compact_clear_kernel, dim3((unsigned)clear), dim3(kPlanThreads), 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "compact clear launch");
    const int64_t marks = std::max<int64_t>(1, std::min<int64_t>((p.entries + kPlanThreads - 1) / kPlanThreads, pool->num_sms));
    e = launch_pdl(compact_mark_kernel, dim3((unsigned)marks), dim3(kPlanThreads), 0, s, p);
    launches = 2;
  }
  if (e != cudaSuccess) return cuda_fail(e, "compact plan launch");
  e = prepare_kernel(pool, compact_move_kernel, kBulkSmem);
  if (e == cudaSuccess) e = launch_pdl(compact_move_kernel, dim3(movers), dim3(kWorkers * 32), kBulkSmem, s, g, p);
  if (e != cudaSuccess) return cuda_fail(e, "compact move launch");
  pool->last_launches = launches + 1;
  return PKV_OK;
}
