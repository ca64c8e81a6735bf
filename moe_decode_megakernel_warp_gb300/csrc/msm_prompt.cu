// msm_prompt.cu — causal attention of packed prompts (msm_prompt_attention).
//
// One block takes 64 rows of one kv head, a row being one (token, query head of the group)
// pair, token-major, so that the heads of a group share the K and V tiles; four warps of 16
// rows run m16n8k16 products with the running maximum and sum of the softmax in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "msm_device.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kRowsQ = 64, kRowsK = 64, kThreadsP = 128;

struct Bf16 {
  static constexpr uint32_t kExponent = 0x7F80u;
  static __device__ __forceinline__ float value(uint16_t b) { return bf16_to_f32(b); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
struct Fp16 {
  static constexpr uint32_t kExponent = 0x7C00u;
  static __device__ __forceinline__ float value(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Elements of V that are not finite are taken out of the products, where a weight of zero
// would spread them (0 x inf = NaN) to rows that do not see their key, and added to the rows
// that do at the end.  Returns whether the vector had any.
template <class El>
__device__ __forceinline__ bool take_out(uint4& v) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t& w = (&v.x)[i];
    if ((w & El::kExponent) == El::kExponent) {
      w &= 0xFFFF0000u;
      any = true;
    }
    if (((w >> 16) & El::kExponent) == El::kExponent) {
      w &= 0xFFFFu;
      any = true;
    }
  }
  return any;
}

struct Seq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Seq prompt_seq(const PromptAttn& p, int s) {
  Seq r;
  r.q0 = min(max(p.q_starts[s], 0), p.n_q);
  r.nq = max(0, min(max(p.q_starts[s + 1], 0), p.n_q) - r.q0);
  r.k0 = min(max(p.k_starts[s], 0), p.n_k);
  r.nk = max(0, min(max(p.k_starts[s + 1], 0), p.n_k) - r.k0);
  return r;
}

// sequence and tile of tile t of the batch (each warp looks for itself); false: behind the last
__device__ bool find_tile(const PromptAttn& p, int t, int rows, int& seq, int& tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int c = 0; c < p.n_seqs; c += 32) {
    int n = 0;
    if (c + lane < p.n_seqs) n = (prompt_seq(p, c + lane).nq * p.group + rows - 1) / rows;
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, t < before + v);
    if (hit) {
      const int l = __ffs(hit) - 1;
      seq = c + l;
      const int first = __shfl_sync(0xffffffffu, before + v - n, l);
      const int cnt = __shfl_sync(0xffffffffu, n, l);
      tile = cnt - 1 - (t - first);  // the longest rows first
      return true;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  return false;
}

template <class El, int HD>
__global__ void __launch_bounds__(kThreadsP) prompt_kernel(const PromptAttn p) {
  constexpr int S = HD + 8;
  __shared__ __align__(16) uint16_t s_k[kRowsK][S];
  __shared__ __align__(16) uint16_t s_v[kRowsK][S];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
  int seq, tile;
  if (!find_tile(p, blockIdx.x, kRowsQ, seq, tile)) return;
  const Seq sq = prompt_seq(p, seq);
  const int h = blockIdx.y, shift = sq.nk - sq.nq;
  const int row0 = tile * kRowsQ, tok0 = row0 / p.group;
  const int tok1 = min(sq.nq, (row0 + kRowsQ - 1) / p.group + 1);
  const int hi = min(sq.nk, tok1 + shift);  // keys behind the last query's
  const int lo = p.window > 0 ? max(0, tok0 + shift - p.window + 1) : 0;
  // q fragments of rows g and g + 8 of the warp
  int row[2], tok[2], head[2];
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    row[r] = row0 + wid * 16 + g + 8 * r;
    tok[r] = row[r] / p.group;
    head[r] = h * p.group + row[r] % p.group;
    const bool ok = tok[r] < sq.nq;
    const uint16_t* const src = p.q + (int64_t)(sq.q0 + (ok ? tok[r] : 0)) * p.q_token + head[r] * p.q_head;
#pragma unroll
    for (int j = 0; j < HD / 16; ++j) {
      qf[j][r] = ok ? *reinterpret_cast<const uint32_t*>(src + j * 16 + 2 * t) : 0u;
      qf[j][r + 2] = ok ? *reinterpret_cast<const uint32_t*>(src + j * 16 + 2 * t + 8) : 0u;
    }
  }
  float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < HD / 8; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) o[i][q] = 0.f;
  bool taken = false;
  for (int k0 = lo; k0 < hi; k0 += kRowsK) {
    __syncthreads();
    for (int i = tid; i < kRowsK * HD / 8; i += kThreadsP) {
      const int r = i / (HD / 8), c = i % (HD / 8) * 8;
      const bool ok = k0 + r < hi;  // (rows behind the end may hold anything: zeros, since 0 x NaN is NaN)
      const int64_t key = sq.k0 + k0 + r;
      *reinterpret_cast<uint4*>(&s_k[r][c]) =
          ok ? *reinterpret_cast<const uint4*>(p.k + key * p.k_token + h * p.k_head + c) : make_uint4(0, 0, 0, 0);
      uint4 v =
          ok ? *reinterpret_cast<const uint4*>(p.v + key * p.v_token + h * p.v_head + c) : make_uint4(0, 0, 0, 0);
      taken |= take_out<El>(v);
      *reinterpret_cast<uint4*>(&s_v[r][c]) = v;
    }
    __syncthreads();
    float sc[kRowsK / 8][4];
#pragma unroll
    for (int n = 0; n < kRowsK / 8; ++n) {
#pragma unroll
      for (int q = 0; q < 4; ++q) sc[n][q] = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 16; ++j) {
        const uint32_t b0 = *reinterpret_cast<const uint32_t*>(&s_k[n * 8 + g][j * 16 + 2 * t]);
        const uint32_t b1 = *reinterpret_cast<const uint32_t*>(&s_k[n * 8 + g][j * 16 + 2 * t + 8]);
        El::mma(sc[n], qf[j], b0, b1);
      }
    }
    float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kRowsK / 8; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int key = k0 + n * 8 + 2 * t + (q & 1), gap = tok[q >> 1] + shift - key;
        const bool see = gap >= 0 && (p.window == 0 || gap < p.window) && key < hi;
        sc[n][q] = see ? sc[n][q] * p.scale_log2 : -INFINITY;
        x[q >> 1] = fmaxf(x[q >> 1], sc[n][q]);
      }
    float ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      x[r] = fmaxf(x[r], __shfl_xor_sync(0xffffffffu, x[r], 1));
      x[r] = fmaxf(x[r], __shfl_xor_sync(0xffffffffu, x[r], 2));
      const float n = fmaxf(m[r], x[r]);
      const float a = m[r] == n ? 1.f : exp2_fast(m[r] - n);
      m[r] = n;
      ref[r] = n == -INFINITY ? 0.f : n;
      l[r] *= a;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        o[i][2 * r] *= a;
        o[i][2 * r + 1] *= a;
      }
    }
#pragma unroll
    for (int n = 0; n < kRowsK / 8; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sc[n][q] = exp2_fast(sc[n][q] - ref[q >> 1]);
        l[q >> 1] += sc[n][q];
      }
#pragma unroll
    for (int j = 0; j < kRowsK / 16; ++j) {
      const uint32_t a[4] = {El::pack(sc[2 * j][0], sc[2 * j][1]), El::pack(sc[2 * j][2], sc[2 * j][3]),
                             El::pack(sc[2 * j + 1][0], sc[2 * j + 1][1]), El::pack(sc[2 * j + 1][2], sc[2 * j + 1][3])};
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(smem_u32(&s_v[j * 16 + (lane & 15)][i * 16 + (lane >> 4) * 8]), b0, b1, b2, b3);
        El::mma(o[2 * i], a, b0, b1);
        El::mma(o[2 * i + 1], a, b2, b3);
      }
    }
  }
  if (__syncthreads_or(taken)) {
    for (int key = lo; key < hi; ++key) {
      const uint16_t* const src = p.v + (int64_t)(sq.k0 + key) * p.v_token + h * p.v_head;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int gap = tok[q >> 1] + shift - key;
          const uint16_t x = src[i * 8 + 2 * t + (q & 1)];
          if ((x & El::kExponent) == El::kExponent && gap >= 0 && (p.window == 0 || gap < p.window))
            o[i][q] += El::value(x);
        }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (tok[r] >= sq.nq) continue;
    const float inv = tok[r] + shift < 0 ? 0.f : 1.f / l[r];  // no key seen: zeros
    uint16_t* const dst = p.out + (int64_t)(sq.q0 + tok[r]) * p.out_token + head[r] * p.out_head;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
      *reinterpret_cast<uint32_t*>(dst + i * 8 + 2 * t) = El::pack(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
  }
}

template <class El, int HD>
cudaError_t launch(const PromptAttn& p, cudaStream_t s) {
  const int64_t tiles = ((int64_t)p.n_q * p.group + kRowsQ - 1) / kRowsQ + p.n_seqs;
  prompt_kernel<El, HD><<<dim3((unsigned)tiles, p.n_kv_heads), kThreadsP, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttn& p, int dtype, int head_dim, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, s) : launch<Bf16, 128>(p, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, s) : launch<Fp16, 128>(p, s);
}

}  // namespace msm
