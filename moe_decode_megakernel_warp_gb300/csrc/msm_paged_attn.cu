// msm_paged_attn.cu — attention of one new token per sequence over a paged KV cache:
//   out[s, h] = sum_j softmax_j(scale q[s, h] . k[j]) v[j]
// over the rows j of sequence s (the last `window` of them on a sliding-window layer),
// query head h reading kv head h / group.
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
// to 8,192 rows 61 us; one of 200 rows (8 heads on 2 of 64) 7 us.

#include <atomic>

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

// The rows of one sequence that a call reads: [lo, hi), in tiles from base (lo rounded down to
// a chunk).  An item costs its block one unit more than its tiles: finishing it takes about as long
// as a tile (64 sequences of 1 to 8,192 rows: 80 us without that unit, 60 us with it).
struct Rows {
  int lo, hi, base, tiles, units;
};
__device__ __forceinline__ Rows seq_rows(const PagedAttn& p, int s) {
  Rows r;
  const int64_t cap = (int64_t)p.max_pages * p.page_rows;
  r.hi = (int)min((int64_t)max(p.lens[s], 0), cap);
  r.lo = p.window > 0 ? max(0, r.hi - p.window) : 0;
  r.base = r.lo & ~31;
  r.tiles = (r.hi - r.base + kTile - 1) / kTile;
  r.units = r.tiles > 0 ? r.tiles + 1 : 0;
  return r;
}

// The work of one block on one (sequence, head): tiles [ta, tb), rows [first, end).
struct Segment {
  int s, h;
  int lo, end, first;  // rows below lo are not seen
  int ta, tb, tiles;   // its tiles of the item's
  int64_t unit0;       // the batch's unit that holds the item's first tile
};

// Walks the segments of a block's run of units [u, u1) (a whole warp together).  Unit 0 of an item
// has no tile.
struct Walk {
  int64_t u, u1, before;  // before: units of the sequences in front of s
  int s;
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
      g.unit0 = before + (int64_t)g.h * rw.units + 1;
      g.ta = max(0, (int)(u - g.unit0));
      g.tb = (int)min((int64_t)rw.tiles, u1 - g.unit0);
      g.tiles = rw.tiles;
      g.lo = rw.lo;
      g.first = rw.base + g.ta * kTile;
      g.end = min(rw.hi, rw.base + g.tb * kTile);
      u = g.unit0 + g.tb;
      if (g.tb > g.ta) return true;
    }
    return false;
  }
};

template <int HD>
struct Cfg {
  static constexpr int kRowBytes = HD * 2;
  static constexpr int kChunk = HD == 128 ? 16 : 32;          // rows of one warp step: 8 KB of K and V
  static constexpr int kStep = kWarps * kChunk;               // rows of one step of the block
  static constexpr int kStageBytes = 2 * kChunk * kRowBytes;
  // One step on the way while another one is worked on: 64 KB per SM cover the latency, and
  // more of them cost DRAM locality (head_dim 128, 64 sequences of 16,384 rows: two stages
  // 6,736 GB/s, three 6,457).
  static constexpr int kStages = 2;
  static constexpr int kOutStride = HD + 4;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRingBytes + kWarps * kHeads * kOutStride * 4;
};

// 16-byte piece c of row r of a chunk: the permutation keeps the eight lanes of a phase on
// different banks for the K reads (two rows x four pieces) and the V reads (four rows of one
// parity x two pieces) alike
__device__ __forceinline__ int swizzle(int r, int c) { return c ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2); }

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

template <class El, int HD>
__global__ void __launch_bounds__(kThreadsA, kPagedAttnPerSm) paged_attn_kernel(const PagedAttn p) {
  using C = Cfg<HD>;
  constexpr int KB = HD / 32;  // 32-element blocks of a K row
  constexpr int VB = HD / 64;  // 64-element blocks of a V row
  constexpr int kAhead = C::kStages - 1;
  constexpr int kSub = C::kChunk / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_find[2];  // first sequence of the block's run, units before it
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_flag;
  float (*const s_o)[kHeads][C::kOutStride] =
      reinterpret_cast<float (*)[kHeads][C::kOutStride]>(smem + C::kRingBytes);
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
  Walk ahead{u0, u1, s_find[1], (int)s_find[0]};
  Segment fs{};
  int fc = 0;  // the next chunk to fetch: row of its first row; -1: none left
  int page = 0;
  // the page of row lane % kChunk of the next chunk
  auto look = [&]() {
    const int r = fc + lane % C::kChunk;
    page = fc >= 0 && r < fs.end ? p.table[(size_t)fs.s * p.max_pages + r / p.page_rows] : -1;
  };
  // the next chunk of this warp, in this or a later segment
  auto find_chunk = [&]() {
    while (fc < 0 || fc >= fs.end) {
      if (!ahead.next(p, fs)) {
        fc = -1;
        return;
      }
      fc = fs.first + wid * C::kChunk;
    }
  };
  int f_stage = 0;
  bool lost = false;  // a table entry outside the pool
  // fetches a chunk and returns which of its rows take part (0 when none is left)
  auto fetch = [&]() -> uint32_t {
    uint32_t rows = 0;
    if (fc >= 0) {
      const int r = fc + lane % C::kChunk;
      bool ok = r >= fs.lo && r < fs.end;
      if (ok && (page < 0 || page >= p.n_pages)) {
        lost = true;
        ok = false;
      }
      rows = __ballot_sync(0xffffffffu, ok);
      // pool row of row lane % kChunk
      const uint32_t at = ((uint32_t)page * p.n_kv_heads + fs.h) * p.page_rows + r % p.page_rows;
      const uint32_t dst = ring + f_stage * C::kStageBytes;
      constexpr int kPieces = HD / 8, kRowsAtOnce = 32 / kPieces;  // 16-byte pieces of a row
      const int c = lane % kPieces, sub = lane / kPieces;
#pragma unroll
      for (int i = 0; i < C::kChunk / kRowsAtOnce; ++i) {
        const int row = i * kRowsAtOnce + sub;
        const uint32_t pr = __shfl_sync(0xffffffffu, at, row);
        const bool in = rows >> row & 1;
        const size_t off = in ? (size_t)pr * HD + c * 8 : 0;
        const uint32_t d = dst + row * C::kRowBytes + swizzle(row, c) * 16;
        cp_async16(d, p.k + off, in ? 16 : 0);
        cp_async16(d + C::kChunk * C::kRowBytes, p.v + off, in ? 16 : 0);
      }
      f_stage = f_stage + 1 == C::kStages ? 0 : f_stage + 1;
      fc += C::kStep;
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
#pragma unroll
  for (int i = 0; i < kAhead; ++i) queue[i] = fetch();

  Walk walk{u0, u1, s_find[1], (int)s_find[0]};
  Segment sg;
  int stage = 0;
  // q of the group as the B operand: column g = query head, the contraction index in the
  // order of the K reads
  uint4 qf[KB];
  auto load_q = [&]() {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      qf[j] = make_uint4(0u, 0u, 0u, 0u);
      if (g < p.group)
        qf[j] = *reinterpret_cast<const uint4*>(p.q + sg.s * p.q_seq + (sg.h * p.group + g) * p.q_head + j * 32 + t * 8);
    }
  };
  bool more = walk.next(p, sg);
  load_q();
  while (more) {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2t, 2t + 1
    uint32_t seen = 0;  // rows that took part
    float o[HD / 16][4];
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[i][q] = 0.f;
    for (int c0 = sg.first + wid * C::kChunk; c0 < sg.end; c0 += C::kStep) {
      cp_async_wait<kAhead - 1>();
      __syncwarp();
      const uint32_t rows = queue[0];
      seen |= rows;
      const uint32_t kb = ring + stage * C::kStageBytes, vb = kb + C::kChunk * C::kRowBytes;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) queue[i] = queue[i + 1];
      queue[kAhead - 1] = fetch();  // into the stage that the previous step read
      // 16 rows at a time: rows g (sc[0], sc[1]) and g + 8 (sc[2], sc[3]); heads 2t and 2t + 1
      float sc[kSub][4];
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sc[u][q] = 0.f;
        const uint32_t k0 = kb + (u * 16 + g) * C::kRowBytes, k1 = k0 + 8 * C::kRowBytes;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const uint4 a = lds128(k0 + swizzle(g, j * 4 + t) * 16), c = lds128(k1 + swizzle(g, j * 4 + t) * 16);
          El::mma(sc[u], a.x, c.x, a.y, c.y, qf[j].x, qf[j].y);
          El::mma(sc[u], a.z, c.z, a.w, c.w, qf[j].z, qf[j].w);
        }
        const bool ok0 = rows >> (u * 16 + g) & 1, ok1 = rows >> (u * 16 + g + 8) & 1;
        sc[u][0] = ok0 ? sc[u][0] * p.scale_log2 : -INFINITY;
        sc[u][1] = ok0 ? sc[u][1] * p.scale_log2 : -INFINITY;
        sc[u][2] = ok1 ? sc[u][2] * p.scale_log2 : -INFINITY;
        sc[u][3] = ok1 ? sc[u][3] * p.scale_log2 : -INFINITY;
        x0 = fmaxf(x0, fmaxf(sc[u][0], sc[u][2]));
        x1 = fmaxf(x1, fmaxf(sc[u][1], sc[u][3]));
      }
#pragma unroll
      for (int q = 4; q <= 16; q <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, q));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, q));
      }
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        // (with no score above -inf yet there is nothing to scale)
        const float a0 = m0 == n0 ? 1.f : exp2_fast(m0 - n0), a1 = m1 == n1 ? 1.f : exp2_fast(m1 - n1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a1;
          o[i][2] *= a0;
          o[i][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
      }
      const float r0 = (m0 == -INFINITY ? 0.f : m0) - Split<El>::kTop, r1 = (m1 == -INFINITY ? 0.f : m1) - Split<El>::kTop;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const float e0 = exp2_fast(sc[u][0] - r0), e1 = exp2_fast(sc[u][1] - r1), e2 = exp2_fast(sc[u][2] - r0),
                    e3 = exp2_fast(sc[u][3] - r1);
        l0 += e0 + e2;
        l1 += e1 + e3;
        // P as two 16-bit terms for the product; its sum keeps 32 bits
        uint32_t h0, h1, w0, w1;
        Split<El>::split(e0, e1, h0, w0);
        Split<El>::split(e2, e3, h1, w1);
        h0 = transpose8x8(h0);
        h1 = transpose8x8(h1);
        w0 = transpose8x8(w0);
        w1 = transpose8x8(w1);
#pragma unroll
        for (int j = 0; j < VB; ++j) {
          // V rows 2t, 2t + 1, 2t + 8, 2t + 9, elements 8g .. 8g + 7 of the block
          uint4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = 2 * t + (q & 1) + 8 * (q >> 1);
            v[q] = lds128(vb + (u * 16 + i) * C::kRowBytes + swizzle(i, j * 8 + g) * 16);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v0 = (&v[0].x)[i], v1 = (&v[1].x)[i], v2 = (&v[2].x)[i], v3 = (&v[3].x)[i];
            // element 64 j + 8 g + 2 i in row g of the product, the next one in row g + 8
            const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632),
                           a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
            El::mma(o[j * 4 + i], a0, a1, a2, a3, h0, h1);
            El::mma(o[j * 4 + i], a0, a1, a2, a3, w0, w1);
          }
        }
      }
    }

    // the warps' results joined; the next segment's q travels meanwhile
#pragma unroll
    for (int q = 4; q <= 16; q <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, q);
      l1 += __shfl_xor_sync(0xffffffffu, l1, q);
    }
    if (g == 0) {
      s_m[wid][2 * t] = m0;
      s_m[wid][2 * t + 1] = m1;
      s_l[wid][2 * t] = seen ? l0 : kNoKeys;
      s_l[wid][2 * t + 1] = seen ? l1 : kNoKeys;
    }
#pragma unroll
    for (int j = 0; j < VB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = j * 64 + 8 * g + 2 * i;
        *reinterpret_cast<float2*>(&s_o[wid][2 * t][d]) = make_float2(o[j * 4 + i][0], o[j * 4 + i][2]);
        *reinterpret_cast<float2*>(&s_o[wid][2 * t + 1][d]) = make_float2(o[j * 4 + i][1], o[j * 4 + i][3]);
      }
    const Segment done = sg;
    more = walk.next(p, sg);
    if (more) load_q();
    __syncthreads();
    const bool whole = done.ta == 0 && done.tb == done.tiles;
    // a run's first item that began before it goes to the block's slot 0, the last one that
    // goes on behind it to slot 1
    float* const part = p.part + (size_t)(2 * b + (done.ta > 0 ? 0 : 1)) * part_len;
    for (int i = tid; i < p.group * HD / 2; i += kThreadsA) {
      const int hd = i / (HD / 2), d = (i - hd * (HD / 2)) * 2;
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) m = fmaxf(m, s_m[q][hd]);
      const float ref = m == -INFINITY ? 0.f : m;
      float l = kNoKeys, x = 0.f, y = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        // (a NaN sum passes on; a warp without rows has m = -inf and zeros)
        const float f = exp2_fast(s_m[q][hd] - ref);
        const float2 v = *reinterpret_cast<const float2*>(&s_o[q][hd][d]);
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

template <class El, int HD>
cudaError_t launch(const PagedAttn& p, int blocks, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit for this kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<El, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<HD>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  paged_attn_kernel<El, HD><<<blocks, kThreadsA, Cfg<HD>::kSmem, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

size_t paged_attn_workspace(int blocks, int group, int head_dim) {
  return (size_t)2 * blocks * part_floats(group, head_dim) * sizeof(float) + 3 * blocks * sizeof(uint32_t);
}

cudaError_t launch_paged_attn(const PagedAttn& p, int dtype, int head_dim, int blocks, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, blocks, s) : launch<Bf16, 128>(p, blocks, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, blocks, s) : launch<Fp16, 128>(p, blocks, s);
}

}  // namespace msm
