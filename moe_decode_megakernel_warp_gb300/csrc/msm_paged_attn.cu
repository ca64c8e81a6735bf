// msm_paged_attn.cu — attention of one new token per sequence over a paged KV cache:
//   out[s, h] = sum_j softmax_j(scale q[s, h] . k[j]) v[j]
// over the rows j of sequence s (the last `window` of them on a sliding-window layer),
// query head h reading kv head h / group.
//
// Bound by memory: every K and V row is read once, 4 flops per element.  The work is cut
// into tiles of 128 rows of one (sequence, kv head); every block takes an equal, contiguous
// run of the tiles of the whole batch, so ragged lengths and a single long sequence load
// all SMs alike.  A (sequence, head) whose tiles all fall to one block is finished there;
// the others leave partial results (maximum, sum, unnormalised output in 32 bits), at most
// two per block, which a second launch joins.
//
// Inside a block the eight warps take 16 rows each and work without shared memory: with
// S^T = K Q^T the K rows are the A operand of m16n8k16 products (16 rows x up to 8 query
// heads of the group), loaded straight into its registers 16 bytes at a time -- the order
// of the contraction index is free, so lane t of a quad takes 8 consecutive elements for
// two products.  O^T = V^T P^T takes V rows the same way, interleaving pairs of rows with
// byte permutes, and P^T comes out of S^T by an 8 x 8 transpose in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "msm_device.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsA = kWarps * 32;
constexpr int kChunk = 16;               // rows of one warp step
constexpr int kTile = kWarps * kChunk;   // rows of one work unit
constexpr int kHeads = 8;                // columns of the products: query heads of a kv head

struct Bf16 {
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    mma_bf16(d, a0, a1, a2, a3, b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
struct Fp16 {
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    mma_f16(d, a0, a1, a2, a3, b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 ld_row(const uint16_t* p, bool ok) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (ok) v = __ldcs(reinterpret_cast<const uint4*>(p));
  return v;
}

// a partial result in the workspace: item, maxima and sums, outputs
__host__ __device__ constexpr int part_floats(int group, int hd) { return 4 + 2 * kHeads + group * hd; }

struct Rows {  // the rows of one sequence that a call reads
  int lo, hi, base, tiles;  // [lo, hi); base = lo rounded down to a chunk
};
__device__ __forceinline__ Rows seq_rows(const PagedAttn& p, int s) {
  Rows r;
  const int64_t cap = (int64_t)p.max_pages * p.page_rows;
  r.hi = (int)min((int64_t)max(p.lens[s], 0), cap);
  r.lo = p.window > 0 ? max(0, r.hi - p.window) : 0;
  r.base = r.lo & ~(kChunk - 1);
  r.tiles = (r.hi - r.base + kTile - 1) / kTile;
  return r;
}

// kPaged16: page_rows is a multiple of 16, so a warp's 16 rows lie in one page (one table
// look-up per step instead of one per row)
template <class El, int HD, bool kPaged16>
__global__ void __launch_bounds__(kThreadsA, 2) paged_attn_kernel(const PagedAttn p) {
  constexpr int KB = HD / 32;  // 32-element blocks of a K row
  constexpr int VB = HD / 64;  // 64-element blocks of a V row
  constexpr int kOutStride = HD + 4;
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_find[2];  // first sequence of the block's run, tiles before it
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ float s_o[kWarps][kHeads][kOutStride];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = gridDim.x, b = blockIdx.x;
  const int part_len = part_floats(p.group, HD);

  // the batch's tiles and where this block's run begins
  int64_t total = 0;
  for (int c = 0; c < p.n_seqs; c += kThreadsA) {
    int64_t x = c + tid < p.n_seqs ? (int64_t)seq_rows(p, c + tid).tiles * p.n_kv_heads : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) s_sum[wid] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_sum[w];
    __syncthreads();
  }
  // (no more blocks than tiles, so that the parts of an item lie in consecutive blocks)
  const int64_t busy = min((int64_t)G, total);
  const int64_t u0 = b < busy ? total * b / busy : 0, u1 = b < busy ? total * (b + 1) / busy : 0;
  // sequences without rows: zeros, shared out over the blocks
  for (int s = b; s < p.n_seqs; s += G)
    if (seq_rows(p, s).tiles == 0)
      for (int i = tid; i < p.n_kv_heads * p.group * HD; i += kThreadsA)
        p.out[s * p.out_seq + (i / HD) * p.out_head + i % HD] = 0;
  if (tid < 2) p.part[(size_t)(2 * b + tid) * part_len] = __int_as_float(-1);  // no partial result yet
  if (u0 >= u1) return;
  int64_t run = 0;
  for (int c = 0; c < p.n_seqs; c += kThreadsA) {
    const int64_t x = c + tid < p.n_seqs ? (int64_t)seq_rows(p, c + tid).tiles * p.n_kv_heads : 0;
    int64_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) s_sum[wid] = v;
    __syncthreads();
    for (int w = 0; w < wid; ++w) v += s_sum[w];
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += s_sum[w];
    if (run + v - x <= u0 && u0 < run + v) {
      s_find[0] = c + tid;
      s_find[1] = run + v - x;
    }
    __syncthreads();
    run += all;
    if (run > u0) break;
  }
  int s = (int)s_find[0];
  int64_t before = s_find[1];  // tiles of the sequences before s

  for (int64_t u = u0; u < u1;) {
    Rows rw = seq_rows(p, s);
    while (u >= before + (int64_t)rw.tiles * p.n_kv_heads) {
      before += (int64_t)rw.tiles * p.n_kv_heads;
      rw = seq_rows(p, ++s);
    }
    const int h = (int)((u - before) / rw.tiles);
    const int64_t item0 = before + (int64_t)h * rw.tiles;  // first tile of (s, h)
    const int ta = (int)(u - item0), tb = (int)min((int64_t)rw.tiles, u1 - item0);
    const int k_end = min(rw.hi, rw.base + tb * kTile);

    // q of the group as the B operand: column g = query head, the contraction index in the
    // order of the K loads
    uint32_t qf[KB][4];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (g < p.group)
        x = *reinterpret_cast<const uint4*>(p.q + s * p.q_seq + (h * p.group + g) * p.q_head + j * 32 + t * 8);
      qf[j][0] = x.x;
      qf[j][1] = x.y;
      qf[j][2] = x.z;
      qf[j][3] = x.w;
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2t, 2t + 1
    float o[HD / 16][4];
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[i][q] = 0.f;

    const int32_t* const row_tab = p.table + (size_t)s * p.max_pages;
    bool lost = false;  // a table entry outside the pool
    // page of the chunk's first row (kPaged16), or of row c0 + lane % 16
    auto look = [&](int c0) -> int {
      const int r = kPaged16 ? c0 : c0 + (lane & 15);
      return r < k_end ? row_tab[r / p.page_rows] : 0;
    };
    // pool row of the chunk's row 0 (kPaged16) or of row lane % 16; -1: not in the pool
    auto pool_row = [&](int c0, int page) -> int64_t {
      const int r = kPaged16 ? c0 : c0 + (lane & 15);
      if (page < 0 || page >= p.n_pages) {
        lost |= r < k_end && (kPaged16 || r >= rw.lo);
        return -1;
      }
      return ((int64_t)page * p.n_kv_heads + h) * p.page_rows + r % p.page_rows;
    };
    auto row_of = [&](int64_t pr, int i) -> int64_t {  // pool row of the chunk's row i, or -1
      if (kPaged16) return pr < 0 ? pr : pr + i;
      return __shfl_sync(0xffffffffu, pr, i);
    };
    auto seen = [&](int c0, int i, int64_t row) -> bool {
      const int r = c0 + i;
      return r >= rw.lo && r < k_end && row >= 0;
    };
    auto load_k = [&](int c0, int64_t pr, uint4 (&kf)[2][KB], bool (&ok)[2]) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = g + 8 * hf;
        const int64_t row = row_of(pr, i);
        const uint16_t* const src = p.k + row * HD + t * 8;
        ok[hf] = seen(c0, i, row);
#pragma unroll
        for (int j = 0; j < KB; ++j) kf[hf][j] = ld_row(src + j * 32, ok[hf]);
      }
    };

    int c0 = rw.base + ta * kTile + wid * kChunk;
    int64_t pr = -1;
    int page_next = 0;
    uint4 kf[2][KB];
    bool ok[2] = {false, false};
    if (c0 < k_end) {
      pr = pool_row(c0, look(c0));
      load_k(c0, pr, kf, ok);
      if (c0 + kTile < k_end) page_next = look(c0 + kTile);
    }
    while (c0 < k_end) {
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the chunk, elements 8g .. 8g + 7 of each block
      uint4 vf[4][VB];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 2 * t + (q & 1) + 8 * (q >> 1);
        const int64_t row = row_of(pr, i);
        const uint16_t* const src = p.v + row * HD + g * 8;
        const bool see = seen(c0, i, row);
#pragma unroll
        for (int j = 0; j < VB; ++j) vf[q][j] = ld_row(src + j * 64, see);
      }
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        El::mma(sc, kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y, qf[j][0], qf[j][1]);
        El::mma(sc, kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w, qf[j][2], qf[j][3]);
      }
      // rows g (sc[0], sc[1]) and g + 8 (sc[2], sc[3]); heads 2t and 2t + 1
      sc[0] = ok[0] ? sc[0] * p.scale_log2 : -INFINITY;
      sc[1] = ok[0] ? sc[1] * p.scale_log2 : -INFINITY;
      sc[2] = ok[1] ? sc[2] * p.scale_log2 : -INFINITY;
      sc[3] = ok[1] ? sc[3] * p.scale_log2 : -INFINITY;
      // the next chunk's K rows travel while this one's softmax and second product run
      const int cn = c0 + kTile;
      int64_t prn = -1;
      if (cn < k_end) {
        prn = pool_row(cn, page_next);
        load_k(cn, prn, kf, ok);
        if (cn + kTile < k_end) page_next = look(cn + kTile);
      }
      float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
#pragma unroll
      for (int w = 4; w <= 16; w <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
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
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      const float e0 = exp2_fast(sc[0] - r0), e1 = exp2_fast(sc[1] - r1), e2 = exp2_fast(sc[2] - r0),
                  e3 = exp2_fast(sc[3] - r1);
      l0 += e0 + e2;
      l1 += e1 + e3;
      // P rounded to the 16-bit type for the product (a relative error of half a step per
      // weight, as V itself carries); its sum keeps 32 bits
      const uint32_t b0 = transpose8x8(El::pack(e0, e1)), b1 = transpose8x8(El::pack(e2, e3));
#pragma unroll
      for (int j = 0; j < VB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v0 = (&vf[0][j].x)[i], v1 = (&vf[1][j].x)[i], v2 = (&vf[2][j].x)[i], v3 = (&vf[3][j].x)[i];
          // element 64 j + 8 g + 2 i in row g of the product, the next one in row g + 8
          El::mma(o[j * 4 + i], __byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632),
                  __byte_perm(v2, v3, 0x5410), __byte_perm(v2, v3, 0x7632), b0, b1);
        }
      c0 = cn;
      pr = prn;
    }
    if (lost) atomicCAS(p.status, 0, MSM_ERR_INVALID_ARG | (kCallAttention << 8));

    // the warps' results joined
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, w);
      l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    if (g == 0) {
      s_m[wid][2 * t] = m0;
      s_m[wid][2 * t + 1] = m1;
      s_l[wid][2 * t] = l0;
      s_l[wid][2 * t + 1] = l1;
    }
#pragma unroll
    for (int j = 0; j < VB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = j * 64 + 8 * g + 2 * i;
        *reinterpret_cast<float2*>(&s_o[wid][2 * t][d]) = make_float2(o[j * 4 + i][0], o[j * 4 + i][2]);
        *reinterpret_cast<float2*>(&s_o[wid][2 * t + 1][d]) = make_float2(o[j * 4 + i][1], o[j * 4 + i][3]);
      }
    __syncthreads();
    const bool whole = ta == 0 && tb == rw.tiles;
    // a run's first item that began before it goes to the block's slot 0, the last one that
    // goes on behind it to slot 1
    float* const part = p.part + (size_t)(2 * b + (ta > 0 ? 0 : 1)) * part_len;
    for (int i = tid; i < p.group * HD / 2; i += kThreadsA) {
      const int hd = i / (HD / 2), d = (i - hd * (HD / 2)) * 2;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][hd]);
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // (a NaN sum passes on; a warp without rows has m = -inf and zeros)
        const float f = exp2_fast(s_m[w][hd] - ref);
        const float2 v = *reinterpret_cast<const float2*>(&s_o[w][hd][d]);
        l += f * s_l[w][hd];
        x += f * v.x;
        y += f * v.y;
      }
      if (whole) {
        const float inv = 1.f / l;
        *reinterpret_cast<uint32_t*>(p.out + s * p.out_seq + (h * p.group + hd) * p.out_head + d) =
            El::pack(x * inv, y * inv);
      } else {
        *reinterpret_cast<float2*>(part + 4 + 2 * kHeads + hd * HD + d) = make_float2(x, y);
        if (d == 0) {
          part[4 + hd] = m;
          part[4 + kHeads + hd] = l;
        }
      }
    }
    if (!whole && tid == 0) {
      part[0] = __int_as_float(s);
      part[1] = __int_as_float(h);
      part[2] = __int_as_float(tb == rw.tiles);  // the item ends here
    }
    __syncthreads();
    u = item0 + tb;
  }
}

// Joins the partial results: block (b, y) finishes the item that begins in block b's slot 1
// (blocks b + 1, b + 2, ... hold its further parts in slot 0 until one says that it ends
// there), columns [64 y, 64 y + 64) of its group * HD outputs; 16 threads across the
// columns, 16 parts at a time.
constexpr int kJoinCols = 64;
template <class El, int HD>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedAttn p, int G) {
  __shared__ float s_m[16], s_l[16];
  __shared__ float4 s_x[16][kJoinCols / 4];
  __shared__ int s_n;
  pdl_wait();
  const int part_len = part_floats(p.group, HD);
  const int b = blockIdx.x, c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const float* const first = p.part + (size_t)(2 * b + 1) * part_len;
  const int s = __float_as_int(first[0]);
  if (s < 0) return;
  const int h = __float_as_int(first[1]);
  const int col = blockIdx.y * kJoinCols + 4 * c, hd = (int)blockIdx.y * kJoinCols / HD;
  // parts of the item: up to and with the first one that ends it
  if (threadIdx.x == 0) s_n = G;
  __syncthreads();
  for (int i0 = 1; b + i0 < G; i0 += 256) {
    const int i = i0 + (int)threadIdx.x;
    if (b + i < G) {
      const float* const q = p.part + (size_t)(2 * (b + i)) * part_len;
      if (__float_as_int(q[0]) != s || __float_as_int(q[1]) != h) atomicMin(&s_n, i);
      else if (__float_as_int(q[2])) atomicMin(&s_n, i + 1);
    }
    __syncthreads();
    if (s_n <= i0 + 256) break;
  }
  const int n = min(s_n, G - b);
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = r; i < n; i += 16) {
    const float* const q = i == 0 ? first : p.part + (size_t)(2 * (b + i)) * part_len;
    const float mq = q[4 + hd], lq = q[4 + kHeads + hd];
    const float4 v = *reinterpret_cast<const float4*>(q + 4 + 2 * kHeads + col);
    const float mn = fmaxf(m, mq);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float fa = exp2_fast(m - ref), fb = exp2_fast(mq - ref);
    l = l * fa + lq * fb;
    x.x = x.x * fa + v.x * fb;
    x.y = x.y * fa + v.y * fb;
    x.z = x.z * fa + v.z * fb;
    x.w = x.w * fa + v.w * fb;
    m = mn;
  }
  if (c == 0) {
    s_m[r] = m;
    s_l[r] = l;
  }
  s_x[r][c] = x;
  __syncthreads();
  if (r != 0) return;
  float mm = -INFINITY;
#pragma unroll
  for (int i = 0; i < 16; ++i) mm = fmaxf(mm, s_m[i]);
  const float ref = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float f = exp2_fast(s_m[i] - ref);
    const float4 v = s_x[i][c];
    ll += f * s_l[i];
    y.x += f * v.x;
    y.y += f * v.y;
    y.z += f * v.z;
    y.w += f * v.w;
  }
  const float inv = 1.f / ll;
  uint2 w;
  w.x = El::pack(y.x * inv, y.y * inv);
  w.y = El::pack(y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(p.out + s * p.out_seq + (h * p.group + hd) * p.out_head + col % HD) = w;
}

template <class El, int HD>
cudaError_t launch(const PagedAttn& p, int blocks, cudaStream_t s) {
  if (p.page_rows % kChunk == 0) paged_attn_kernel<El, HD, true><<<blocks, kThreadsA, 0, s>>>(p);
  else paged_attn_kernel<El, HD, false><<<blocks, kThreadsA, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(blocks, p.group * HD / kJoinCols);
  lc.blockDim = dim3(256);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, paged_join_kernel<El, HD>, p, blocks);
}

}  // namespace

size_t paged_attn_workspace(int blocks, int group, int head_dim) {
  return (size_t)2 * blocks * part_floats(group, head_dim) * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttn& p, int dtype, int head_dim, int blocks, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, blocks, s) : launch<Bf16, 128>(p, blocks, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, blocks, s) : launch<Fp16, 128>(p, blocks, s);
}

}  // namespace msm
