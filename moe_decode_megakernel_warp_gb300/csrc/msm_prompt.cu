// msm_prompt.cu — causal attention of packed prompts (msm_prompt_attention):
//   out[i, h] = sum_j softmax_j(scale q[i, h] . k[j]) v[j]   over the keys that i sees.
//
// A row is one (token, query head of the group) pair, token-major, so that the heads of a
// group share the K and V tiles and a tile spans few tokens (few masked scores).  One block
// takes 256 rows of one kv head as two tiles of 128, one per softmax warpgroup, and walks the
// 128-key tiles that its rows see from the last to the first:
//   S = Q K^T and O += P V run on tcgen05 (kind::f16), Q, K and V in shared memory by TMA,
//   S, P and O in tensor memory.  While one tile's softmax runs, the tensor cores work on
//   the other's: P0 V, Q0 K(next), P1 V, Q1 K(next), ...
//   A softmax thread owns a row (128 scores in registers), so its maximum and sum need no
//   exchange.  P takes the place of S (16-bit, half its columns).  O is only rescaled when a
//   row's maximum has grown by more than 2^8 since the last time (P stays below 2^8, well
//   inside fp16); S(j + 1) being there means that P(j) V is done, the products of a block being issued
//   and completed in order, so the thread may then change O itself.
// Warps 0-7: softmax; 8: product issue; 9: TMA loads; 10, 11: finite check of V.
//
// A weight of zero does not stop an infinite or NaN element of V (0 x inf = NaN), and a
// masked score has such a weight.  In key tiles that some row sees only in part, warps 10 and
// 11 therefore take these elements out before the product; the rows that do see their keys
// get them back at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "msm_device.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kRows = 128;                   // rows of a tile: the M of the products
constexpr int kKeys = 128;                   // keys of a tile
constexpr int kBlockRows = 2 * kRows;
constexpr int kPromptThreads = 384;
constexpr int kBoxBytes = kRows * 128;       // 128 rows x 64 elements, one swizzle span wide
// Registers: 384 threads start with 168; warps 8-11 give up 64 each, warps 0-7 take 32
// (256 x 200 + 128 x 104 = 384 x 168).
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
constexpr float kGrow = 8.0f;  // log2 of the largest unnormalised weight
constexpr uint64_t kWaitNs = 2000000000ull;

struct Bf16 {
  static constexpr bool kBf16 = true;
  static constexpr uint32_t kExponent = 0x7F80u;
  static __device__ __forceinline__ float value(uint16_t b) { return bf16_to_f32(b); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
struct Fp16 {
  static constexpr bool kBf16 = false;
  static constexpr uint32_t kExponent = 0x7C00u;
  static __device__ __forceinline__ float value(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

template <int HD>
struct Cfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = HD == 128 ? 5 : 10;  // K and V tiles in flight: 160 KB
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
};

struct Maps {
  CUtensorMap q, k, v;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Waits for a phase of a barrier, at most kWaitNs: false (and `dead` set, which ends the other
// warps' waits) when it did not come.
__device__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i % 64 == 0) {
      if (*dead) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitNs) {
        *dead = 1;
        return false;
      }
    }
  }
}

template <int kCount>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kCount));
}
template <int kCount>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCount));
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
__device__ bool find_tile(const PromptAttn& p, int t, int& seq, int& tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int c = 0; c < p.n_seqs; c += 32) {
    int n = 0;
    if (c + lane < p.n_seqs) n = (prompt_seq(p, c + lane).nq * p.group + kBlockRows - 1) / kBlockRows;
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
      tile = cnt - 1 - (t - first);  // those with the most keys first
      return true;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  return false;
}

// the block's work
struct Work {
  int q0, nq, k0, shift, window;
  int row0, tok0, tok1;  // first row, its token, one past the last token
  int hi;                // one past the last key that any row sees
  int t_lo, n;           // first key tile, their number
  bool two;              // the second tile has rows
  __device__ int tile(int j) const { return t_lo + n - 1 - j; }
  // does some row see only a part of tile j?
  __device__ bool partial(int j) const {
    const int a = tile(j) * kKeys;
    return a + kKeys - 1 > tok0 + shift || (window > 0 && a < tok1 + shift - window);
  }
};

template <class El, int HD>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ Maps maps, const PromptAttn p) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t b_q[2], b_full[C::kStages], b_empty[C::kStages], b_clean[C::kStages], b_s[2], b_p[2],
      b_o[2], b_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_taken;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int seq, tile;
  const int h = blockIdx.x % p.n_kv_heads;
  if (!find_tile(p, blockIdx.x / p.n_kv_heads, seq, tile)) return;
  Work w;
  {
    const Seq sq = prompt_seq(p, seq);
    w.q0 = sq.q0;
    w.nq = sq.nq;
    w.k0 = sq.k0;
    w.shift = sq.nk - sq.nq;
    w.window = p.window;
    w.row0 = tile * kBlockRows;
    w.tok0 = w.row0 / p.group;
    w.tok1 = min(sq.nq, w.tok0 + kBlockRows / p.group);
    w.hi = max(0, w.tok1 + w.shift);
    const int lo = p.window > 0 ? max(0, w.tok0 + w.shift - p.window + 1) : 0;
    w.t_lo = lo / kKeys;
    w.n = w.hi > 0 ? (w.hi + kKeys - 1) / kKeys - w.t_lo : 0;
    w.two = w.row0 + kRows < sq.nq * p.group;
  }
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_q = smem;
  uint8_t* const s_kv = smem + 2 * C::kTileBytes;

  if (w.n == 0) {  // no row sees a key
    for (int r = wid; r < kBlockRows; r += kPromptThreads / 32) {
      const int tok = (w.row0 + r) / p.group;
      if (tok >= w.nq) break;
      uint16_t* const dst = p.out + (int64_t)(w.q0 + tok) * p.out_token + (h * p.group + r % p.group) * p.out_head;
      if (lane < HD / 8) reinterpret_cast<uint4*>(dst)[lane] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  if (wid == 8) tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&b_q[t], 1);
      mbar_init(&b_s[t], 1);
      mbar_init(&b_p[t], 4);
      mbar_init(&b_o[t], 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
      mbar_init(&b_clean[i], 2);
    }
    mbar_init(&b_drain, 1);
    s_dead = s_taken = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_shared();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t t_s[2] = {tmem, tmem + 128}, t_o[2] = {tmem + 256, tmem + 256 + HD};
  volatile int* const dead = &s_dead;

  if (wid >= 8) {
    set_max_regs_down<kOtherRegs>();
    if (wid == 9) {
      // ---- loads: Q0, K(0), Q1, then V(j), K(j + 1), ... through the ring
      if (lane == 0) {
        int issued = 0;
        auto load_q = [&](int t) {
          mbar_expect_tx(&b_q[t], C::kTileBytes);
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(s_q + t * C::kTileBytes + x * kBoxBytes, &maps.q, x * 64, 0, h,
                        w.q0 + w.tok0 + t * (kRows / p.group), &b_q[t]);
        };
        load_q(0);
        for (int i = 0; i < 2 * w.n; ++i) {
          const int st = i % C::kStages;
          if (i >= C::kStages && !wait_bar(&b_empty[st], (i / C::kStages + 1) & 1, dead)) break;
          mbar_expect_tx(&b_full[st], C::kTileBytes);
          const CUtensorMap* const map = i & 1 ? &maps.v : &maps.k;
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_3d(s_kv + st * C::kTileBytes + x * kBoxBytes, map, x * 64, h, w.k0 + w.tile(i >> 1) * kKeys,
                        &b_full[st]);
          issued = i + 1;
          if (i == 0 && w.two) load_q(1);
        }
        if (*dead) {  // nothing of this block may be on its way when it ends
          int never = 0;
          wait_bar(&b_q[0], 0, &never);
          if (w.two) wait_bar(&b_q[1], 0, &never);
          for (int i = max(0, issued - C::kStages); i < issued; ++i)
            wait_bar(&b_full[i % C::kStages], (i / C::kStages) & 1, &never);
        }
      }
    } else if (wid == 8) {
      // ---- products
      if (lane == 0) {
        const uint32_t i_s = idesc_f16(El::kBf16, p.scale_log2 < 0.f, false, kKeys);
        const uint32_t i_o = idesc_f16(El::kBf16, false, true, HD);
        auto full = [&](int i) { return wait_bar(&b_full[i % C::kStages], (i / C::kStages) & 1, dead); };
        auto scores = [&](int t, int i) {  // S = Q K^T
          const uint32_t a = smem_u32(s_q + t * C::kTileBytes), b = smem_u32(s_kv + (i % C::kStages) * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t off = (k / 4) * kBoxBytes + (k % 4) * 32;
            mma_f16_ss(t_s[t], sdesc_k_sw128(a + off), sdesc_k_sw128(b + off), i_s, k > 0);
          }
          tc_commit(&b_s[t]);
        };
        auto values = [&](int t, int i, bool first) {  // O += P V
          const uint32_t b = smem_u32(s_kv + (i % C::kStages) * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_f16_ts(t_o[t], t_s[t] + k * 8, sdesc_mn_sw128(b + k * 2048, kBoxBytes), i_o, !first || k > 0);
        };
        uint32_t clean_phase = 0;
        bool ok = wait_bar(&b_q[0], 0, dead) && full(0);
        if (ok) {
          tc_fence_after();
          scores(0, 0);
          if (w.two) {
            ok = wait_bar(&b_q[1], 0, dead);
            if (ok) scores(1, 0);
          }
          tc_commit(&b_empty[0]);
        }
        for (int j = 0; ok && j < w.n; ++j) {
          const int iv = 2 * j + 1, ik = 2 * j + 2, st = iv % C::kStages;
          ok = full(iv);
          if (ok && w.partial(j)) {
            ok = wait_bar(&b_clean[st], clean_phase >> st & 1, dead);
            clean_phase ^= 1u << st;
          }
          if (!ok) break;
          for (int t = 0; t < (w.two ? 2 : 1); ++t) {
            if (!(ok = wait_bar(&b_p[t], j & 1, dead))) break;
            tc_fence_after();
            values(t, iv, j == 0);
            if (j + 1 < w.n) {
              if (t == 0 && !(ok = full(ik))) break;
              scores(t, ik);
            } else {
              tc_commit(&b_o[t]);
            }
          }
          tc_commit(&b_empty[st]);
          if (j + 1 < w.n) tc_commit(&b_empty[ik % C::kStages]);
        }
        if (*dead) {  // nor any product
          int never = 0;
          tc_commit(&b_drain);
          wait_bar(&b_drain, 0, &never);
        }
      }
    } else {
      // ---- finite check of the V tiles that some row sees in part
      constexpr uint32_t kE = El::kExponent, kLow = kE & (~kE + 1u);  // exponent field, its lowest bit
      for (int j = 0; j < w.n; ++j) {
        if (!w.partial(j)) continue;
        const int i = 2 * j + 1, st = i % C::kStages;
        if (!__all_sync(0xffffffffu, wait_bar(&b_full[st], (i / C::kStages) & 1, dead))) break;
        uint4* const v = reinterpret_cast<uint4*>(s_kv + st * C::kTileBytes);
        bool any = false;
#pragma unroll 4
        for (int c = (wid - 10) * 32 + lane; c < C::kTileBytes / 16; c += 64) {
          const uint4 x = v[c];
          // an exponent of all ones carries into the sign's place
          const uint32_t m = kE * 0x10001u, a = kLow * 0x10001u;
          const uint32_t bad = (((x.x & m) + a) | ((x.y & m) + a) | ((x.z & m) + a) | ((x.w & m) + a)) & 0x80008000u;
          if (bad) {
            any = true;
            uint16_t* const e = reinterpret_cast<uint16_t*>(v + c);
            for (int q = 0; q < 8; ++q)
              if ((e[q] & kE) == kE) e[q] = 0;
          }
        }
        if (any) {
          s_taken = 1;
          fence_proxy_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_clean[st], 1);
      }
    }
  } else {
    // ---- softmax: thread = row
    set_max_regs_up<kSoftmaxRegs>();
    const int t = wid >> 2;
    if (t == 0 || w.two) {
      const int row = w.row0 + t * kRows + (wid & 3) * 32 + lane;
      const int tok = row / p.group, head = h * p.group + row % p.group;
      const int last = tok + w.shift;                                // the last key that the row sees
      const int first = w.window > 0 ? max(0, last - w.window + 1) : 0;  // and the first one
      const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
      const uint32_t ts = t_s[t] + lanes, to = t_o[t] + lanes;
      // (a negative scale negates Q in the product; a scale of zero must still leave -inf x scale = -inf)
      const float scale = fmaxf(fabsf(p.scale_log2), 1e-30f);
      float m = -INFINITY;
      uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      bool ok = true;
      for (int j = 0; j < w.n; ++j) {
        ok = __all_sync(0xffffffffu, wait_bar(&b_s[t], j & 1, dead));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s[c]);
        tmem_ld_wait();
        if (w.partial(j)) {
          const int a = first - w.tile(j) * kKeys, b = last - w.tile(j) * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i < a || c * 32 + i > b) s[c][i] = 0xFF800000u;
        }
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            x[c] = fmaxf(x[c], fmaxf(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])));
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (j == 0) {
          m = mx;
        } else {
          const bool grow = (mx - m) * scale > kGrow;
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? exp2_fast((m - mx) * scale) : 1.f;
            if (grow) m = mx;
            const uint64_t ff = pair(f, f);
            l2[0] = fma2(l2[0], ff, pair(0.f, 0.f));
            l2[1] = fma2(l2[1], ff, pair(0.f, 0.f));
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(to + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(to + c * 16, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m * scale;
        const uint64_t sc2 = pair(scale, scale), neg2 = pair(neg, neg);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), sc2, neg2), e0, e1);
            e0 = exp2_fast(e0);
            e1 = exp2_fast(e1);
            l2[i & 1] = add2(l2[i & 1], pair(e0, e1));
            // rounded to the 16-bit type for the product with V; the sum keeps 32 bits
            pk[i] = El::pack(e0, e1);
          }
          tmem_st16(ts + c * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_p[t], 1);
      }
      ok = ok && __all_sync(0xffffffffu, wait_bar(&b_o[t], 0, dead));
      tc_fence_after();
      float l0, l1;
      unpair(add2(l2[0], l2[1]), l0, l1);
      // no key seen: zeros; a wait that ran out: NaN
      const float inv = !ok ? NAN : last < 0 ? 0.f : 1.f / (l0 + l1);
      const bool taken = *(volatile int*)&s_taken != 0;
      uint16_t* const dst = p.out + (int64_t)(w.q0 + tok) * p.out_token + head * p.out_head;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(to + c * 32, o);
        tmem_ld_wait();
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
        if (taken && tok < w.nq) {
          for (int j = 0; j < w.n; ++j) {
            if (!w.partial(j)) continue;
            const int a = max(first, w.tile(j) * kKeys), b = min(last, w.tile(j) * kKeys + kKeys - 1);
            for (int key = a; key <= b; ++key) {
              const uint16_t* const v = p.v + (int64_t)(w.k0 + key) * p.v_token + h * p.v_head + c * 32;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((v[i] & El::kExponent) == El::kExponent) f[i] += El::value(v[i]);
            }
          }
        }
        if (tok < w.nq) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(dst + c * 32 + i) =
                make_uint4(El::pack(f[i], f[i + 1]), El::pack(f[i + 2], f[i + 3]), El::pack(f[i + 4], f[i + 5]),
                           El::pack(f[i + 6], f[i + 7]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (wid == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};

cudaError_t encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
  PFN_cuTensorMapEncodeTiled_v12000 f = g_encode.load(std::memory_order_relaxed);
  if (!f) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qr;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr);
    if (e != cudaSuccess) return e;
    if (!fn || qr != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    g_encode.store(f, std::memory_order_relaxed);
  }
  *out = f;
  return cudaSuccess;
}

// rows [tokens][heads][HD] as boxes of 64 elements; Q's heads are split into (group, kv head)
template <class El, int HD>
cudaError_t launch(const PromptAttn& p, cudaStream_t s) {
  const int64_t tiles = ((int64_t)p.n_q * p.group + kBlockRows - 1) / kBlockRows + p.n_seqs;
  const int64_t blocks = tiles * p.n_kv_heads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  Maps maps;
  const CUtensorMapDataType type = El::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  auto make = [&](CUtensorMap* m, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
    return encode(m, type, rank, const_cast<void*>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t qd[4] = {HD, (cuuint64_t)p.group, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_q};
  const cuuint64_t qs[3] = {(cuuint64_t)p.q_head * 2, (cuuint64_t)p.q_head * 2 * p.group, (cuuint64_t)p.q_token * 2};
  const cuuint32_t qb[4] = {64, (cuuint32_t)p.group, 1, (cuuint32_t)(kRows / p.group)};
  bool ok = make(&maps.q, 4, p.q, qd, qs, qb);
  // (without keys no block loads any: the maps then only have to be valid)
  const cuuint64_t kd[3] = {HD, (cuuint64_t)p.n_kv_heads, (cuuint64_t)(p.n_k > 0 ? p.n_k : 1)};
  const cuuint64_t ks[2] = {(cuuint64_t)p.k_head * 2, (cuuint64_t)p.k_token * 2};
  const cuuint64_t vs[2] = {(cuuint64_t)p.v_head * 2, (cuuint64_t)p.v_token * 2};
  const cuuint32_t kb[3] = {64, 1, kKeys};
  ok = ok && make(&maps.k, 3, p.n_k > 0 ? p.k : p.q, kd, ks, kb) && make(&maps.v, 3, p.n_k > 0 ? p.v : p.q, kd, vs, kb);
  if (!ok) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit for this kernel is set
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    // the warps' register shares must add up to what a block starts with, or they would wait
    // for registers that never come
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, prompt_kernel<El, HD>)) != cudaSuccess) return e;
    if (at.numRegs * kPromptThreads < 256 * kSoftmaxRegs + (kPromptThreads - 256) * kOtherRegs)
      return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(prompt_kernel<El, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  prompt_kernel<El, HD><<<(unsigned)blocks, kPromptThreads, Cfg<HD>::kSmem, s>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttn& p, int dtype, int head_dim, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, s) : launch<Bf16, 128>(p, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, s) : launch<Fp16, 128>(p, s);
}

}  // namespace msm
