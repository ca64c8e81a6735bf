// msm_paged_attn.cu — attention of one new token per sequence over a paged KV cache:
//   out[s, h] = sum_j softmax_j(scale q[s, h] . k[j]) v[j]
// over the rows j of sequence s (the last `window` of them on a sliding-window layer, and with sinks
// the first few), query head h reading kv head h / group.  A cache in 8 bits (kHeld8) holds e4m3 codes with a
// scale for a block of rows: k[j] = ks_j k8[j], v[j] = vs_j v8[j].
//
// Bound by memory: every K and V row is read once, 4 flops per element.  The work is cut
// into tiles of 64 rows of one (sequence, kv head); every block (two per SM) takes an equal,
// contiguous run of the tiles of the whole batch, so ragged lengths and a single long
// sequence load all SMs alike.  A (sequence, head) whose tiles all fall to one block is
// finished there; the others leave partial results (maximum, sum, unnormalised output in 32
// bits), at most two per block, which the last block of them to arrive joins in the order of
// the tiles, so the result does not depend on which one that is.
//
// Inside a block the four warps take 16 (head_dim 64: 32) rows at a time each, every warp with
// a ring of its own in shared memory that cp.async keeps filled across the ends of items (rows
// outside the sequence or its window are filled with zeros, never read).  With S^T = K Q^T the K
// rows are the A operand of m16n8k16 products (16 rows x up to 8 query heads of the group), read
// 16 bytes at a time -- the order of the contraction index is free, so lane t of a quad takes
// 8 consecutive elements for two products.  O^T = V^T P^T takes V rows the same way,
// interleaving pairs of rows with byte permutes, and P^T comes out of S^T by an 8 x 8
// transpose in registers.  (Register loads without the rings: 5,610 GB/s where these reach
// 6,550; one block of eight warps per SM is as fast on long sequences and 1.7 times slower on short ones.)
//
// On one GB300 (6,691 GB/s measured copy rate), 32 query heads on 8 kv heads of 128, bf16: 64
// sequences of 4,096 rows 165 us (6,500 GB/s from DRAM), one of 131,071 rows 89 us, 64 of 1
// to 8,192 rows 61 us; one of 200 rows (8 heads on 2 of 64) 7 us.  128 streams of 700 to 8,192 rows on a window
// of 2,048 and 64 sinks, fp16: 139 us (6,200 GB/s).
//
// 8 bits: half the bytes, so the instructions per row weigh twice.  A code becomes fp16 by one conversion
// instruction for two (exactly: fp16 has every e4m3 value), on its way from shared memory into the same
// products; V's codes of two rows are interleaved by a byte permutation first, so that one conversion gives the
// pair that the product wants.  K's scale multiplies the score, V's the weight.  Weights times V's scale
// can lie anywhere, so they are relative to a maximum of their own, that of score + log2(scale), and the
// output is brought back to the scores' maximum at the end of a segment.  An item of few tiles is done by one
// warp alone, without the block's barriers (PagedAttn::solo_tiles).  Measured: 131,071 rows 55 us (5,000
// GB/s: 38 us at 7,000 GB/s between 3 us of start and 6 us of join), 64 sequences of 1 to 8,192 rows 34 us (3,300
// GB/s; on a window of 2,048 with 64 sinks 27 us), 512 sequences of 30 rows 27 us.  These have pages of 64 rows and
// more: 32 rows that lie in one page are fetched with addresses that differ by constants.  Pages of 16 rows never
// allow that: 131,071 rows 56 us, the ragged batch 36, and 128 streams of 700 to 8,192 rows on a window of 2,048
// with 64 sinks 95 where pages of 64 rows take 86.  The ragged batch is bound by the ends of its 512 items and by the chain of
// a step's products, exchanges and exponentials with two warps per scheduler: leaving out the conversions changed
// nothing, leaving out the loads 5 %.  Three blocks per SM: 58 and 33 us, and with chunks of 16 rows 64 and 39.

#include <atomic>
#include <type_traits>

#include "msm_attn.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreadsA = kWarps * 32;
constexpr int kTile = kWarps * 16;       // rows of a tile
constexpr int kHeads = 8;                // columns of the products: query heads of a kv head

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 16 bytes to shared memory, zeros where `bytes` is 0
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// The sum of a row's weights where no key took part (every row that a sequence reads lies on pages
// outside the pool): -0, which stays -0 through sums of such and products with factors, and which
// becomes 0 with any other sum -- a sum of 0 is that of scores that are all -inf.
constexpr float kNoKeys = -0.f;
// 1 / l, and 0 where no key took part
__device__ __forceinline__ float inverse_sum(float l) { return __float_as_uint(l) == 0x80000000u ? 0.f : 1.f / l; }

// Weights as the B operand.  One 16-bit term is off by up to half a step (2^-8, 2^-11), and equal
// weights all err the same way, so a weight is split into hi + lo: off by at most 3 half steps
// squared.  Beside the reads the second product costs nothing (64 sequences of 4,096 rows 165 us
// either way, one of 2,000 rows 11.3 us).  hi is the weight made smaller by a step before it is
// rounded, so that lo is above 0, too (down to weights of 2^-125, fp16 2^-28 of the largest): a lo
// of 0 or below would make NaN of the infinite value of a key that is seen.
template <class El>
struct Split {
  static constexpr float kLess = El::kBf16 ? 1.f - 0x1p-7f : 1.f - 0x1p-10f;
  // log2 of the largest weight.  fp16 ends at 2^-25 (half its smallest step): with weights up to
  // 2^14 that is 2^-39 of the largest, so that the many small ones of a long context still count.
  static constexpr float kTop = El::kBf16 ? 0.f : 14.f;
  static __device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = El::pack(a * kLess, b * kLess);
    lo = El::pack(a - El::value((uint16_t)(hi & 0xFFFFu)), b - El::value((uint16_t)(hi >> 16)));
  }
};

// a partial result in the workspace: maxima, sums, outputs
__host__ __device__ constexpr int part_floats(int group, int hd) { return 2 * kHeads + group * hd; }

// The rows of one sequence that a call reads: the sinks [0, first) and the window [lo, hi), in
// tiles.  Places count them through: without sinks a place is its row, from base (lo rounded down to a
// chunk) to hi.  With sinks in front of the window the tiles that hold them come first, from place 0,
// and the places from `pad` on are the rows `skip` further on, from base.  (Where those tiles reach the
// window there is nothing to skip.)  An item costs its block `finish` units more than its tiles, what
// finishing it takes (64 sequences of 1 to 8,192 rows: 80 us without, 60 us with one unit).
struct Rows {
  int lo, hi, base, tiles, units;  // hi, base: places
  int first, pad, skip;
};
__device__ __forceinline__ Rows seq_rows(const PagedAttn& p, int s) {
  Rows r;
  const int64_t cap = (int64_t)p.max_pages * p.page_rows;
  r.hi = (int)min((int64_t)max(p.lens[s], 0), cap);
  r.lo = p.window > 0 ? max(0, r.hi - p.window) : 0;
  r.base = r.lo & ~31;
  r.first = min(p.sinks, r.lo);
  r.pad = r.skip = 0;
  if (r.first > 0) {
    r.pad = (r.first + kTile - 1) / kTile * kTile;
    r.skip = max(0, r.base - r.pad);
    r.hi -= r.skip;
    r.base = 0;
  }
  r.tiles = (r.hi - r.base + kTile - 1) / kTile;
  r.units = r.tiles > p.solo_tiles ? r.tiles + p.finish : r.tiles > 0 ? r.tiles + 1 : 0;
  return r;
}

// The work of one block on one (sequence, head): tiles [ta, tb), places [first, end).
struct Segment {
  int s, h;
  int lo, sinks;       // rows below lo are not seen, but for the first `sinks`
  int pad, skip;       // as in Rows
  int end, first;
  int ta, tb, tiles;   // its tiles of the item's
  int solo;            // 8 bits, a short item: the warp that does all of it; else -1
  int64_t unit0;       // the batch's unit that holds the item's first tile
  __device__ __forceinline__ int row(int place) const { return place < pad ? place : place + skip; }
  __device__ __forceinline__ bool sees(int row) const { return row >= lo || row < sinks; }
};

// Walks the segments of a block's run of units [u, u1) (a whole warp together).  The first units of an
// item, `finish` of them, have no tile.  With kSolo short items go to one warp each, in turn.
template <bool kSolo>
struct Walk {
  int64_t u, u1, before;  // before: units of the sequences in front of s
  int s;
  int solos;              // items of a warp so far
  __device__ bool next(const PagedAttn& p, Segment& g) {
    while (u < u1) {
      Rows rw = seq_rows(p, s);
      if (u >= before + (int64_t)rw.units * p.n_kv_heads) {
        // the sequence that holds u, 32 at a time (most slots of a batch may be empty)
        const int lane = threadIdx.x & 31;
        for (;; s += 32) {
          const int64_t x = s + lane < p.n_seqs ? (int64_t)seq_rows(p, s + lane).units * p.n_kv_heads : 0;
          int64_t v = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, u < before + v);
          const int l = hit ? __ffs(hit) - 1 : 31;
          before += __shfl_sync(0xffffffffu, hit ? v - x : v, l);
          if (hit) {
            s += l;
            break;
          }
          if (s + 32 >= p.n_seqs) return false;  // (lengths that changed during the call)
        }
        rw = seq_rows(p, s);
      }
      g.s = s;
      g.h = (int)((u - before) / rw.units);
      g.unit0 = before + (int64_t)g.h * rw.units + (rw.units - rw.tiles);
      g.ta = max(0, (int)(u - g.unit0));
      g.tb = (int)min((int64_t)rw.tiles, u1 - g.unit0);
      g.tiles = rw.tiles;
      g.lo = rw.lo;
      g.sinks = rw.first;
      g.pad = rw.pad;
      g.skip = rw.skip;
      g.first = rw.base + g.ta * kTile;
      g.end = min(rw.hi, rw.base + g.tb * kTile);
      u = g.unit0 + g.tb;
      g.solo = kSolo && g.tiles <= p.solo_tiles && g.ta == 0 && g.tb == g.tiles ? solos++ % kWarps : -1;
      if (g.tb > g.ta) return true;
    }
    return false;
  }
};

template <int HD, bool kHeld8>
struct Cfg {
  static constexpr int kRowBytes = HD * (kHeld8 ? 1 : 2);
  static constexpr int kChunk = HD == 128 && !kHeld8 ? 16 : 32;  // rows of one warp step: 8 KB of K and V (8 bits of 64: 4 KB)
  static constexpr int kStep = kWarps * kChunk;               // rows of one step of the block
  static constexpr int kStageBytes = 2 * kChunk * kRowBytes;
  // One step on the way while another one is worked on: 64 KB per SM cover the latency, and
  // more of them cost DRAM locality (head_dim 128, 64 sequences of 16,384 rows: two stages
  // 6,736 GB/s, three 6,457).
  static constexpr int kStages = HD == 64 && kHeld8 ? 3 : 2;
  static constexpr int kOutStride = HD + 4;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kOutHeads = kHeld8 ? 4 : kHeads;  // heads whose results the warps put together at a time
  static constexpr int kSmem = kRingBytes + kWarps * kOutHeads * kOutStride * 4;
};

// Where 16-byte piece c of row r of a chunk stands: the permutation keeps the lanes of a phase on
// different banks for the K reads (two rows x four pieces) and the V reads (four rows of one
// parity x two pieces) alike.  Rows of 64 bytes share a line of 128 in pairs.
template <int kRowBytes>
__device__ __forceinline__ int at_piece(int r, int c) {
  if constexpr (kRowBytes == 64) return (r >> 1) * 128 + ((((r & 1) << 2) + c) ^ (((r >> 1) & 3) << 1)) * 16;
  else return r * kRowBytes + (c ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) * 16;
}
// two e4m3 values (the low or the high half of x) as two fp16, which hold every one of them
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The scales of a row of a cache in 8 bits: K's, and V's as f 2^e.  e is a float, -inf for a scale of 0.
struct RowScale {
  float k, f, e;
};
__device__ __forceinline__ RowScale row_scale(float k, float v) {
  RowScale s;
  const bool tiny = fabsf(v) < 0x1p-126f;
  const uint32_t b = __float_as_uint(tiny ? v * 0x1p64f : v), x = b >> 23 & 255u;
  s.k = k;
  s.f = x == 255u ? NAN : __uint_as_float((b & 0x807FFFFFu) | 0x3F800000u);
  s.e = x == 0u ? -INFINITY : (float)((int)x - (tiny ? 127 + 64 : 127));
  return s;
}

// Parts of an item, in the order of its tiles: part i stands in slot 1 of block b0 (i = 0) or
// in slot 0 of block b0 + i.  Joins parts i0, i0 + step, ... (n of them, at most kJoinGroup
// unless `step` is above 1) and writes the output, or a joined part in the place of the
// first one.
constexpr int kJoinGroup = 16;
constexpr int kJoinLoads = 16;
template <class El, int HD>
__device__ void join_parts(const PagedAttn& p, int b0, int i0, int step, int n, int s, int h, bool final,
                           float* s_m, float* s_l) {
  const int part_len = part_floats(p.group, HD);
  auto part = [&](int k) -> float* {
    const int i = i0 + k * step;
    return p.part + (size_t)(2 * (b0 + i) + (i == 0 ? 1 : 0)) * part_len;
  };
  for (int c = threadIdx.x; c < p.group * HD / 4; c += kThreadsA) {  // float4 columns
    const int hd = 4 * c / HD;
    float m = -INFINITY, l = kNoKeys;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += kJoinLoads) {
      float mq[kJoinLoads], lq[kJoinLoads];
      float4 v[kJoinLoads];
#pragma unroll
      for (int q = 0; q < kJoinLoads; ++q) {
        mq[q] = -INFINITY;
        lq[q] = kNoKeys;
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + q < n) {
          const float* const a = part(k0 + q);
          mq[q] = __ldcg(a + hd);
          lq[q] = __ldcg(a + kHeads + hd);
          v[q] = __ldcg(reinterpret_cast<const float4*>(a + 2 * kHeads) + c);
        }
      }
      float mn = m;
#pragma unroll
      for (int q = 0; q < kJoinLoads; ++q) mn = fmaxf(mn, mq[q]);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float fa = exp2_fast(m - ref);
      l *= fa;
      x.x *= fa;
      x.y *= fa;
      x.z *= fa;
      x.w *= fa;
#pragma unroll
      for (int q = 0; q < kJoinLoads; ++q) {
        const float f = exp2_fast(mq[q] - ref);
        l += lq[q] * f;
        x.x += v[q].x * f;
        x.y += v[q].y * f;
        x.z += v[q].z * f;
        x.w += v[q].w * f;
      }
      m = mn;
    }
    if (final) {
      const float inv = inverse_sum(l);
      uint2 o;
      o.x = El::pack(x.x * inv, x.y * inv);
      o.y = El::pack(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(p.out + s * p.out_seq + (h * p.group + hd) * p.out_head + 4 * c % HD) = o;
    } else {
      reinterpret_cast<float4*>(part(0) + 2 * kHeads)[c] = x;
      if (4 * c % HD == 0) {
        s_m[hd] = m;
        s_l[hd] = l;
      }
    }
  }
  if (!final) {
    __syncthreads();  // every column has read the first part's maxima and sums
    if ((int)threadIdx.x < p.group) {
      part(0)[threadIdx.x] = s_m[threadIdx.x];
      part(0)[kHeads + threadIdx.x] = s_l[threadIdx.x];
    }
  }
}

// true for the block that arrives last of n at a counter (which it leaves at zero); what the
// others wrote before they arrived is then visible to it
__device__ bool arrive_last(uint32_t* counter, int n, int* s_flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(counter, 1u) == (uint32_t)n - 1u;
    if (last) *counter = 0u;
    *s_flag = last;
  }
  __syncthreads();
  const bool last = *s_flag != 0;
  if (last) __threadfence();
  return last;
}

template <class El, int HD, bool kHeld8>
__global__ void __launch_bounds__(kThreadsA, kHeld8 ? kQPagedAttnPerSm : kPagedAttnPerSm) paged_attn_kernel(const PagedAttn p) {
  using C = Cfg<HD, kHeld8>;
  // 8-bit rows become fp16 on their way into the products (exactly), and so do q and the weights
  using Mul = typename std::conditional<kHeld8, Fp16, El>::type;
  constexpr int KB = HD / 32;  // 32-element blocks of a K row
  constexpr int VB = HD / 64;  // 64-element blocks of a V row
  constexpr int kAhead = C::kStages - 1;
  constexpr int kSub = C::kChunk / 16;
  constexpr float kSumTop = kHeld8 ? 0.f : Split<Mul>::kTop;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_find[2];  // first sequence of the block's run, units before it
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_flag;
  float (*const s_o)[C::kOutHeads][C::kOutStride] =
      reinterpret_cast<float (*)[C::kOutHeads][C::kOutStride]>(smem + C::kRingBytes);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = gridDim.x, b = blockIdx.x;
  const int part_len = part_floats(p.group, HD);
  const uint32_t ring = smem_u32(smem) + wid * C::kStages * C::kStageBytes;

  // the batch's units: a prefix over the sequences when every thread has one, else their sum
  // first (the prefix is then taken up to the block's run only)
  int64_t total = 0, mine = 0, upto = 0;  // this thread's sequence's units, and with those in front
  for (int c = tid; c < p.n_seqs; c += kThreadsA) mine += (int64_t)seq_rows(p, c).units * p.n_kv_heads;
  {
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) s_sum[wid] = v;
    __syncthreads();
    upto = v;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      if (q < wid) upto += s_sum[q];
      total += s_sum[q];
    }
    __syncthreads();
  }
  if (tid < 2) s_find[tid] = 0;
  // (no more blocks than units, so that the parts of an item lie in consecutive blocks)
  const int64_t busy = min((int64_t)G, total);
  const int64_t u0 = b < busy ? total * b / busy : 0, u1 = b < busy ? total * (b + 1) / busy : 0;
  // sequences without rows: zeros, shared out over the blocks
  for (int s = b; s < p.n_seqs; s += G)
    if (seq_rows(p, s).tiles == 0)
      for (int i = tid; i < p.n_kv_heads * p.group * HD; i += kThreadsA)
        p.out[s * p.out_seq + (i / HD) * p.out_head + i % HD] = 0;
  if (u0 >= u1) return;
  __syncthreads();
  if (p.n_seqs <= kThreadsA) {
    if (upto - mine <= u0 && u0 < upto) {
      s_find[0] = tid;
      s_find[1] = upto - mine;
    }
  } else {
    int64_t run = 0;
    for (int c = 0; run <= u0 && c < p.n_seqs; c += kThreadsA) {
      const int64_t x = c + tid < p.n_seqs ? (int64_t)seq_rows(p, c + tid).units * p.n_kv_heads : 0;
      int64_t v = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) s_sum[wid] = v;
      __syncthreads();
      v += run;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        if (q < wid) v += s_sum[q];
        run += s_sum[q];
      }
      if (v - x <= u0 && u0 < v) {
        s_find[0] = c + tid;
        s_find[1] = v - x;
      }
      __syncthreads();
    }
  }
  __syncthreads();

  // ---- loads: every warp keeps kAhead chunks of its own on the way, across the ends of items
  Walk<kHeld8> ahead{u0, u1, s_find[1], (int)s_find[0], 0};
  Segment fs{};
  int fc = 0;  // the next chunk to fetch: place of its first row; -1: none left
  int page = 0;
  // the page of row lane % kChunk of the next chunk
  auto look = [&]() {
    const int r = fc + lane % C::kChunk;
    page = fc >= 0 && r < fs.end ? p.table[(size_t)fs.s * p.max_pages + p.by_page.of(fs.row(r))] : -1;
  };
  // the next chunk of this warp, in this or a later segment
  auto find_chunk = [&]() {
    while (fc < 0 || fc >= fs.end) {
      if (!ahead.next(p, fs)) {
        fc = -1;
        return;
      }
      fc = fs.first + wid * C::kChunk;
      if (kHeld8 && fs.solo >= 0) fc = fs.solo == wid ? fs.first : fs.end;
    }
  };
  int f_stage = 0;
  bool lost = false;  // a table entry outside the pool
  // fetches a chunk and returns which of its rows take part (0 when none is left)
  auto fetch = [&](float2& rs) -> uint32_t {
    uint32_t rows = 0;
    if (fc >= 0) {
      const int place = fc + lane % C::kChunk, r = fs.row(place);
      bool ok = fs.sees(r) && place < fs.end;
      if (ok && (page < 0 || page >= p.n_pages)) {
        lost = true;
        ok = false;
      }
      rows = __ballot_sync(0xffffffffu, ok);
      // pool row of row lane % kChunk
      const uint32_t head = (uint32_t)page * p.n_kv_heads + fs.h, in_page = r - p.by_page.of(r) * p.page_rows;
      const uint32_t at = head * p.page_rows + in_page;
      if constexpr (kHeld8) {
        const uint32_t i = head * p.page_blocks + p.by_block.of(in_page);
        // (as they are loaded: what is made of them waits for the step that uses them)
        rs = make_float2(0.f, 0.f);
        if (ok) rs = make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
      }
      const uint32_t dst = ring + f_stage * C::kStageBytes;
      constexpr int kPieces = C::kRowBytes / 16, kRowsAtOnce = 32 / kPieces;  // 16-byte pieces of a row
      const int c = lane % kPieces, sub = lane / kPieces;
      bool run = false;  // 8 bits: are all rows there, one behind the other (in one page)?
      if constexpr (kHeld8) {
        const uint32_t at0 = __shfl_sync(0xffffffffu, at, 0);
        run = __all_sync(0xffffffffu, ok && at == at0 + (uint32_t)lane);
      }
      if (run) {  // addresses that differ by constants (a third of the fetch's instructions)
        const size_t off = (size_t)(at - lane) * C::kRowBytes + lane * 16;
        const char *const k0 = static_cast<const char*>(p.k) + off, *const v0 = static_cast<const char*>(p.v) + off;
        // (the permutation depends on the parity of i at most)
        const uint32_t d[2] = {dst + at_piece<C::kRowBytes>(sub, c),
                               dst + at_piece<C::kRowBytes>(kRowsAtOnce + sub, c) - 512};
#pragma unroll
        for (int i = 0; i < C::kChunk / kRowsAtOnce; ++i) {
          cp_async16(d[i & 1] + i * 512, k0 + i * 512, 16);
          cp_async16(d[i & 1] + i * 512 + C::kChunk * C::kRowBytes, v0 + i * 512, 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kChunk / kRowsAtOnce; ++i) {
          const int row = i * kRowsAtOnce + sub;
          const uint32_t pr = __shfl_sync(0xffffffffu, at, row);
          const bool in = rows >> row & 1;
          const size_t off = in ? (size_t)pr * C::kRowBytes + c * 16 : 0;
          const uint32_t d = dst + at_piece<C::kRowBytes>(row, c);
          cp_async16(d, static_cast<const char*>(p.k) + off, in ? 16 : 0);
          cp_async16(d + C::kChunk * C::kRowBytes, static_cast<const char*>(p.v) + off, in ? 16 : 0);
        }
      }
      f_stage = f_stage + 1 == C::kStages ? 0 : f_stage + 1;
      fc += kHeld8 && fs.solo >= 0 ? C::kChunk : C::kStep;
      find_chunk();
      look();
    }
    cp_async_commit();
    return rows;
  };
  fc = -1;
  find_chunk();
  look();
  uint32_t queue[kAhead];
  float2 scales[kAhead] = {};  // of row `lane`: K's, V's
#pragma unroll
  for (int i = 0; i < kAhead; ++i) queue[i] = fetch(scales[i]);

  Walk<kHeld8> walk{u0, u1, s_find[1], (int)s_find[0], 0};
  Segment sg;
  int stage = 0;
  // q of the group as the B operand: column g = query head, the contraction index in the
  // order of the K reads
  uint4 qf[KB];
  float q0 = 1.f, q1 = 1.f;  // what the products with q of heads 2t, 2t + 1 are times too small
  auto load_q = [&]() {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      qf[j] = make_uint4(0u, 0u, 0u, 0u);
      // (8 bits: 16 consecutive elements of a K row a lane, in blocks of 64)
      const int at = kHeld8 ? (j / 2) * 64 + t * 16 + (j & 1) * 8 : j * 32 + t * 8;
      if (g < p.group) qf[j] = *reinterpret_cast<const uint4*>(p.q + sg.s * p.q_seq + (sg.h * p.group + g) * p.q_head + at);
    }
    if constexpr (kHeld8 && El::kBf16) {
      // bf16 to fp16: the head's largest finite element to 2^14 .. 2^15 by a power of two.  Elements down to 2^-31
      // of it stay exact, and what is lost of smaller ones is 2^-39 of it at most.
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = ((&qf[j].x)[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
          most = x < El::kExponent ? max(most, x) : most;
        }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // (elements below 2^-98 keep fewer bits: the factor has to be a number)
      const int up = most ? min(112, 127 + 14 - (int)(most >> 7)) : 0;
      const float f = __uint_as_float((uint32_t)(127 + up) << 23), back = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t& x = (&qf[j].x)[i];
          x = Fp16::pack(El::value((uint16_t)(x & 0xFFFFu)) * f, El::value((uint16_t)(x >> 16)) * f);
        }
      q0 = __shfl_sync(0xffffffffu, back, 8 * t);
      q1 = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
  };
  // the next segment that this warp has a part in
  auto next_segment = [&]() {
    bool any;
    do any = walk.next(p, sg);
    while (kHeld8 && any && sg.solo >= 0 && sg.solo != wid);
    return any;
  };
  bool more = next_segment();
  if (more) load_q();
  while (more) {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2t, 2t + 1
    // 8 bits: the largest score + log2 of V's scale.  What V is multiplied with is relative to this one.
    float v0 = -INFINITY, v1 = -INFINITY;
    uint32_t seen = 0;  // rows that took part
    float o[HD / 16][4];
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[i][q] = 0.f;
    const bool solo = kHeld8 && sg.solo >= 0;
    for (int c0 = sg.first + (solo ? 0 : wid * C::kChunk); c0 < sg.end; c0 += solo ? C::kChunk : C::kStep) {
      cp_async_wait<kAhead - 1>();
      __syncwarp();
      const uint32_t rows = queue[0];
      const RowScale rs = row_scale(scales[0].x, scales[0].y);
      seen |= rows;
      const uint32_t kb = ring + stage * C::kStageBytes, vb = kb + C::kChunk * C::kRowBytes;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) {
        queue[i] = queue[i + 1];
        scales[i] = scales[i + 1];
      }
      queue[kAhead - 1] = fetch(scales[kAhead - 1]);  // into the stage that the previous step read
      // 16 rows at a time: rows g (sc[0], sc[1]) and g + 8 (sc[2], sc[3]); heads 2t and 2t + 1
      float sc[kSub][4];
      float f_a[kSub], f_b[kSub], e_a[kSub], e_b[kSub];  // V's scales of rows g and g + 8
      float x0 = -INFINITY, x1 = -INFINITY, y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sc[u][q] = 0.f;
        const int ra = u * 16 + g, rb = ra + 8;
        const bool ok0 = rows >> ra & 1, ok1 = rows >> rb & 1;
        if constexpr (kHeld8) {
#pragma unroll
          for (int j = 0; j < HD / 64; ++j) {
            const uint4 a = lds128(kb + at_piece<C::kRowBytes>(ra, j * 4 + t)),
                        c = lds128(kb + at_piece<C::kRowBytes>(rb, j * 4 + t));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t aw = (&a.x)[i], cw = (&c.x)[i];
              const uint4& q = qf[2 * j + (i >> 1)];
              Mul::mma(sc[u], e4m3_lo(aw), e4m3_lo(cw), e4m3_hi(aw), e4m3_hi(cw), i & 1 ? q.z : q.x, i & 1 ? q.w : q.y);
            }
          }
          const float ka = __shfl_sync(0xffffffffu, rs.k, ra), kc = __shfl_sync(0xffffffffu, rs.k, rb);
          f_a[u] = __shfl_sync(0xffffffffu, rs.f, ra);
          f_b[u] = __shfl_sync(0xffffffffu, rs.f, rb);
          e_a[u] = __shfl_sync(0xffffffffu, rs.e, ra);
          e_b[u] = __shfl_sync(0xffffffffu, rs.e, rb);
          sc[u][0] = sc[u][0] * q0 * ka;
          sc[u][1] = sc[u][1] * q1 * ka;
          sc[u][2] = sc[u][2] * q0 * kc;
          sc[u][3] = sc[u][3] * q1 * kc;
        } else {
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            const uint4 a = lds128(kb + at_piece<C::kRowBytes>(ra, j * 4 + t)),
                        c = lds128(kb + at_piece<C::kRowBytes>(rb, j * 4 + t));
            Mul::mma(sc[u], a.x, c.x, a.y, c.y, qf[j].x, qf[j].y);
            Mul::mma(sc[u], a.z, c.z, a.w, c.w, qf[j].z, qf[j].w);
          }
        }
        sc[u][0] = ok0 ? sc[u][0] * p.scale_log2 : -INFINITY;
        sc[u][1] = ok0 ? sc[u][1] * p.scale_log2 : -INFINITY;
        sc[u][2] = ok1 ? sc[u][2] * p.scale_log2 : -INFINITY;
        sc[u][3] = ok1 ? sc[u][3] * p.scale_log2 : -INFINITY;
        x0 = fmaxf(x0, fmaxf(sc[u][0], sc[u][2]));
        x1 = fmaxf(x1, fmaxf(sc[u][1], sc[u][3]));
        if constexpr (kHeld8) {
          y0 = fmaxf(y0, fmaxf(sc[u][0] + e_a[u], sc[u][2] + e_b[u]));
          y1 = fmaxf(y1, fmaxf(sc[u][1] + e_a[u], sc[u][3] + e_b[u]));
        }
      }
#pragma unroll
      for (int q = 4; q <= 16; q <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, q));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, q));
        if constexpr (kHeld8) {
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, q));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, q));
        }
      }
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float w0 = fmaxf(v0, y0), w1 = fmaxf(v1, y1);
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1 || (kHeld8 && (w0 > v0 || w1 > v1)))) {
        // (with no score above -inf yet there is nothing to scale)
        const float a0 = m0 == n0 ? 1.f : exp2_fast(m0 - n0), a1 = m1 == n1 ? 1.f : exp2_fast(m1 - n1);
        const float b0 = !kHeld8 ? a0 : v0 == w0 ? 1.f : exp2_fast(v0 - w0);
        const float b1 = !kHeld8 ? a1 : v1 == w1 ? 1.f : exp2_fast(v1 - w1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          o[i][0] *= b0;
          o[i][1] *= b1;
          o[i][2] *= b0;
          o[i][3] *= b1;
        }
        m0 = n0;
        m1 = n1;
        v0 = w0;
        v1 = w1;
      }
      // what scores are relative to in the sum, and for their product with V
      const float r0 = (m0 == -INFINITY ? 0.f : m0) - kSumTop, r1 = (m1 == -INFINITY ? 0.f : m1) - kSumTop;
      const float s0 = (v0 == -INFINITY ? 0.f : v0) - Split<Mul>::kTop + 1.f,
                  s1 = (v1 == -INFINITY ? 0.f : v1) - Split<Mul>::kTop + 1.f;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        float e0 = exp2_fast(sc[u][0] - r0), e1 = exp2_fast(sc[u][1] - r1), e2 = exp2_fast(sc[u][2] - r0),
              e3 = exp2_fast(sc[u][3] - r1);
        l0 += e0 + e2;
        l1 += e1 + e3;
        if constexpr (kHeld8) {
          // weight x V's scale, at most 2^14 (the scale's power of two is in the exponent: neither factor can leave
          // the range)
          e0 = exp2_fast(sc[u][0] + e_a[u] - s0) * f_a[u];
          e1 = exp2_fast(sc[u][1] + e_a[u] - s1) * f_a[u];
          e2 = exp2_fast(sc[u][2] + e_b[u] - s0) * f_b[u];
          e3 = exp2_fast(sc[u][3] + e_b[u] - s1) * f_b[u];
        }
        // P as two 16-bit terms for the product; its sum keeps 32 bits
        uint32_t h0, h1, w0, w1;
        Split<Mul>::split(e0, e1, h0, w0);
        Split<Mul>::split(e2, e3, h1, w1);
        h0 = transpose8x8(h0);
        h1 = transpose8x8(h1);
        w0 = transpose8x8(w0);
        w1 = transpose8x8(w1);
        if constexpr (kHeld8) {
          // V rows 2t, 2t + 1, 2t + 8, 2t + 9, elements HD / 8 g .. + HD / 8
          uint32_t v[4][HD / 32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = u * 16 + 2 * t + (q & 1) + 8 * (q >> 1);
            if constexpr (HD == 128) {
              const uint4 x = lds128(vb + at_piece<C::kRowBytes>(i, g));
              v[q][0] = x.x, v[q][1] = x.y, v[q][2] = x.z, v[q][3] = x.w;
            } else {
              const uint2 x = lds64(vb + at_piece<C::kRowBytes>(i, g >> 1) + (g & 1) * 8);
              v[q][0] = x.x, v[q][1] = x.y;
            }
          }
#pragma unroll
          for (int i = 0; i < HD / 32; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // elements 4 i + 2 half and the next one of two rows, then of the other two
              const uint32_t a = __byte_perm(v[0][i], v[1][i], half ? 0x7362 : 0x5140),
                             c = __byte_perm(v[2][i], v[3][i], half ? 0x7362 : 0x5140);
              const uint32_t a0 = e4m3_lo(a), a1 = e4m3_hi(a), a2 = e4m3_lo(c), a3 = e4m3_hi(c);
              Mul::mma(o[2 * i + half], a0, a1, a2, a3, h0, h1);
              Mul::mma(o[2 * i + half], a0, a1, a2, a3, w0, w1);
            }
        } else {
#pragma unroll
          for (int j = 0; j < VB; ++j) {
            // V rows 2t, 2t + 1, 2t + 8, 2t + 9, elements 8g .. 8g + 7 of the block
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = lds128(vb + at_piece<C::kRowBytes>(u * 16 + 2 * t + (q & 1) + 8 * (q >> 1), j * 8 + g));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v0 = (&v[0].x)[i], v1 = (&v[1].x)[i], v2 = (&v[2].x)[i], v3 = (&v[3].x)[i];
              // element 64 j + 8 g + 2 i in row g of the product, the next one in row g + 8
              const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632),
                             a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
              Mul::mma(o[j * 4 + i], a0, a1, a2, a3, h0, h1);
              Mul::mma(o[j * 4 + i], a0, a1, a2, a3, w0, w1);
            }
          }
        }
      }
    }
    if constexpr (kHeld8) {
      // the output relative to the scores' maximum, as its sum is (two factors: neither leaves the range)
      const float h0 = v0 == -INFINITY ? 0.f : exp2_fast((v0 - Split<Mul>::kTop + 1.f - m0) * 0.5f),
                  h1 = v1 == -INFINITY ? 0.f : exp2_fast((v1 - Split<Mul>::kTop + 1.f - m1) * 0.5f);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        o[i][0] = o[i][0] * h0 * h0;
        o[i][1] = o[i][1] * h1 * h1;
        o[i][2] = o[i][2] * h0 * h0;
        o[i][3] = o[i][3] * h1 * h1;
      }
    }

    // the warps' results joined; the next segment's q travels meanwhile
#pragma unroll
    for (int q = 4; q <= 16; q <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, q);
      l1 += __shfl_xor_sync(0xffffffffu, l1, q);
    }
    if (solo) {  // all of the item: no other warp to wait for
      const float inv0 = inverse_sum(seen ? l0 : kNoKeys), inv1 = inverse_sum(seen ? l1 : kNoKeys);
      uint16_t* const to = p.out + sg.s * p.out_seq + (sg.h * p.group + 2 * t) * p.out_head + HD / 8 * g;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        if (2 * t < p.group) *reinterpret_cast<uint32_t*>(to + 2 * i) = El::pack(o[i][0] * inv0, o[i][2] * inv0);
        if (2 * t + 1 < p.group)
          *reinterpret_cast<uint32_t*>(to + p.out_head + 2 * i) = El::pack(o[i][1] * inv1, o[i][3] * inv1);
      }
      more = next_segment();
      if (more) load_q();
      continue;
    }
    if (g == 0) {
      s_m[wid][2 * t] = m0;
      s_m[wid][2 * t + 1] = m1;
      s_l[wid][2 * t] = seen ? l0 : kNoKeys;
      s_l[wid][2 * t + 1] = seen ? l1 : kNoKeys;
    }
    auto put = [&](int h0) {  // of heads h0 .. h0 + kOutHeads - 1
      if (C::kOutHeads < kHeads && (2 * t < h0 || 2 * t >= h0 + C::kOutHeads)) return;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const int d = kHeld8 ? HD / 8 * g + 2 * i : i / 4 * 64 + 8 * g + 2 * (i % 4);
        *reinterpret_cast<float2*>(&s_o[wid][2 * t - h0][d]) = make_float2(o[i][0], o[i][2]);
        *reinterpret_cast<float2*>(&s_o[wid][2 * t - h0 + 1][d]) = make_float2(o[i][1], o[i][3]);
      }
    };
    put(0);
    const Segment done = sg;
    more = next_segment();
    if (more) load_q();
    __syncthreads();
    const bool whole = done.ta == 0 && done.tb == done.tiles;
    // a run's first item that began before it goes to the block's slot 0, the last one that
    // goes on behind it to slot 1
    float* const part = p.part + (size_t)(2 * b + (done.ta > 0 ? 0 : 1)) * part_len;
    for (int h0 = 0; h0 < p.group; h0 += C::kOutHeads) {
      if (h0 > 0) {
        __syncthreads();
        put(h0);
        __syncthreads();
      }
      for (int i = tid; i < min(p.group - h0, C::kOutHeads) * HD / 2; i += kThreadsA) {
        const int hd = h0 + i / (HD / 2), d = i % (HD / 2) * 2;
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) m = fmaxf(m, s_m[q][hd]);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = kNoKeys, x = 0.f, y = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
          // (a NaN sum passes on; a warp without rows has m = -inf and zeros)
          const float f = exp2_fast(s_m[q][hd] - ref);
          const float2 v = *reinterpret_cast<const float2*>(&s_o[q][hd - h0][d]);
          l += f * s_l[q][hd];
          x += f * v.x;
          y += f * v.y;
        }
        if (whole) {
          const float inv = inverse_sum(l);
          *reinterpret_cast<uint32_t*>(p.out + done.s * p.out_seq + (done.h * p.group + hd) * p.out_head + d) =
              El::pack(x * inv, y * inv);
        } else {
          *reinterpret_cast<float2*>(part + 2 * kHeads + hd * HD + d) = make_float2(x, y);
          if (d == 0) {
            part[hd] = m;
            part[kHeads + hd] = l;
          }
        }
      }
    }
    if (!whole) {
      // the blocks that hold the item's first and last tile; the last one to arrive joins the
      // parts, groups of kJoinGroup first when there are more
      const int b0 = (int)(((done.unit0 + 1) * busy - 1) / total);
      const int n = (int)(((done.unit0 + done.tiles) * busy - 1) / total) - b0 + 1;
      const int k = (b - b0) / kJoinGroup, groups = (n + kJoinGroup - 1) / kJoinGroup;
      const int in_group = min(kJoinGroup, n - k * kJoinGroup);
      // (counters: one of the item that a block begins, one for the groups of that item, one of the
      // group whose first part is the block's slot 0)
      if (arrive_last(p.counters + (k == 0 ? b0 : 2 * G + b0 + k * kJoinGroup), in_group, &s_flag)) {
        join_parts<El, HD>(p, b0, k * kJoinGroup, 1, in_group, done.s, done.h, groups == 1,
                           s_m[0], s_l[0]);
        if (groups > 1 && arrive_last(p.counters + G + b0, groups, &s_flag))
          join_parts<El, HD>(p, b0, 0, kJoinGroup, groups, done.s, done.h, true, s_m[0], s_l[0]);
      }
    }
    __syncthreads();
  }
  if (lost) atomicCAS(p.status, 0, MSM_ERR_INVALID_ARG | (kCallAttention << 8));
}

template <class El, int HD, bool kHeld8>
cudaError_t launch(const PagedAttn& p, int blocks, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit for this kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<El, HD, kHeld8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<HD, kHeld8>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  paged_attn_kernel<El, HD, kHeld8><<<blocks, kThreadsA, Cfg<HD, kHeld8>::kSmem, s>>>(p);
  return cudaGetLastError();
}
template <class El>
cudaError_t launch_as(const PagedAttn& p, int head_dim, int blocks, cudaStream_t s) {
  if (p.k_scales) return head_dim == 64 ? launch<El, 64, true>(p, blocks, s) : launch<El, 128, true>(p, blocks, s);
  return head_dim == 64 ? launch<El, 64, false>(p, blocks, s) : launch<El, 128, false>(p, blocks, s);
}
}  // namespace

size_t paged_attn_workspace(int blocks, int group, int head_dim) {
  return (size_t)2 * blocks * part_floats(group, head_dim) * sizeof(float) + 3 * blocks * sizeof(uint32_t);
}

cudaError_t launch_paged_attn(const PagedAttn& p, int dtype, int head_dim, int blocks, cudaStream_t s) {
  return dtype == MSM_BF16 ? launch_as<Bf16>(p, head_dim, blocks, s) : launch_as<Fp16>(p, head_dim, blocks, s);
}

}  // namespace msm
