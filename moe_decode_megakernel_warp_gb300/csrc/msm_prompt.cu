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
//   exchange.  P takes the place of S (16-bit, half its columns).  P is computed with the
//   maximum that the row had before the tile; only when the tile's own is larger by more than
//   a factor 2^12 O is rescaled and P computed again.
//   S(j + 1) being there means that P(j) V is done, the products of a block being issued
//   and completed in order, so the thread may then change O itself.
// Warps 0-7: softmax; 8, 10: products of a tile each; 9: TMA loads; 11: finite check of V.
//
// A weight of zero does not stop an infinite or NaN element of V (0 x inf = NaN), and a
// masked score has such a weight.  In key tiles that some row sees only in part, warp 11
// therefore takes these elements out before the product; the rows that do see their keys
// get them back at the end.
//
// Bound by the chain of one tile's softmax (1,000 cycles) and its products (1,260 cycles; 1,024
// at the tensor cores' rate -- Q K^T takes all of shared memory's bandwidth, which the TMA
// writes share), two tiles of which overlap: about 2,900 cycles for 256 rows x 128 keys, 2,048 of
// them products.  On one GB300 (1,926 TFLOP/s measured cuBLAS burst), 32 query heads on 8 kv
// heads of 128, bf16: 16,384 tokens 1.39 ms alone (1,580 TFLOP/s) and 1.50 in a row (power), 2,048
// tokens 36 us, 32,768 tokens on a window of 2,048 0.83 ms (1,290 TFLOP/s: two of 17 key tiles are
// masked, 800 cycles each, and the end of a piece of work, every 17, takes 4,500).  At head_dim 64
// the chain is what bounds it still more: 16,384 tokens 1.23 ms (895 TFLOP/s), some 2,740 cycles a
// step of which the products need 1,024; tensor pipe 34 %, exponentials 34 %, issue 41 %.  Tried
// and slower: P handed over in two or four parts (+5, +13 %), results written by four more warps
// (+5 %; fewer registers for the softmax) or through shared memory with four stages of the ring
// instead of five (+4 %), 192 or 208 registers (+7, +2 %).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "msm_attn.cuh"
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
constexpr uint64_t kWaitNs = 2000000000ull;

constexpr float kGrow = 12.0f;  // log2 of how much a row's maximum may be above the one that it works with
// log2 of the weight of a score that equals the maximum that a row works with.  fp16 ends at 2^16 and
// rounds to 0 from 2^-25 on, so weights up to 2^15 keep three bits more of the small ones: down to
// 2^-28 of the largest.  More of them for less growth costs time: 2^-32 and a growth of 2^8 10 %
// on a window of 2,048 (828 us for 32,768 tokens to 905), 2^-29 and 2^11 1 % at head_dim 64.
template <class El>
constexpr float kTop = El::kBf16 ? 0.f : 3.f;

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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 32 bytes at once: the threads of a warp write different rows, so a store's cost is its number of
// separate sectors (32 bytes each)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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

__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* dead) {
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

// Waits for a phase of a barrier, at most kWaitNs: false (and `dead` set, which ends the other
// warps' waits) when it did not come.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, dead);
}

// bits 0 .. n
__device__ __forceinline__ uint32_t bits_upto(int n) { return n < 0 ? 0u : n >= 31 ? 0xFFFFFFFFu : (2u << n) - 1u; }

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

// A warp's place in the batch, in shared memory (registers that last through the softmax cost 2 %)
struct Place {
  int round;
  int c, before;  // first sequence of the 32 looked at last, tiles of the sequences in front of it
};

// Finds the sequence and the tile of the batch's tile t (each warp for itself); false: behind the
// last tile.  t must not fall from call to call: the search goes on where the last one ended.
// The tiles of 32 sequences at a time are listed by their level, the tiles of tokens in front of their
// end (cached ones too), highest first: that is by the keys that they see, the most first (four prompts of
// 2,048 tokens 132 us, listed sequence by sequence 154).  Where the window makes tiles alike, or there is
// one sequence, they are listed sequence by sequence: neighbours share keys, and there is nothing to
// search (12 resumed prompts on a window of 2,048 170 us, by level 175; the one windowed batch measured.
// One sequence with more keys than the window decides it for its 32, so a window that hides few keys of long
// ones gives the order by level up as well).
__device__ bool find_tile(const PromptAttn& p, volatile Place* place, int t, int& seq, int& tile) {
  const int lane = threadIdx.x & 31;
  int c = place->c, before = place->before;
  for (; c < p.n_seqs; c += 32) {
    int n = 0, off = 0, keys = 0;  // a sequence has the levels off .. off + n - 1
    if (c + lane < p.n_seqs) {
      const Seq sq = prompt_seq(p, c + lane);
      n = (sq.nq * p.group + kBlockRows - 1) / kBlockRows;
      off = max(0, sq.nk - sq.nq) * p.group / kBlockRows;
      keys = sq.nk;
    }
    const int all = __reduce_add_sync(0xffffffffu, n);
    if (t < before + all) {
      const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
      const bool alike = __any_sync(0xffffffffu, p.window > 0 && keys > p.window);
      bool it;  // is it this lane's sequence?
      if ((some & (some - 1)) == 0 || alike) {
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        const int r = t - before - (v - n);
        it = r >= 0 && r < n;
        tile = n - 1 - r;
      } else {
        // the level that holds tile t - before: `above` tiles are at higher ones
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, off + n), above = 0;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1, up = __reduce_add_sync(0xffffffffu, max(0, min(n, off + n - mid)));
          if (t - before < up) {
            lo = mid;
          } else {
            hi = mid;
            above = up;
          }
        }
        const bool has = off <= lo && lo < off + n;
        const uint32_t in = __ballot_sync(0xffffffffu, has);
        it = has && __popc(in & ((1u << lane) - 1)) == t - before - above;
        tile = lo - off;
      }
      const int l = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
      seq = c + l;
      tile = __shfl_sync(0xffffffffu, tile, l);
      if (lane == 0) {
        place->c = c;
        place->before = before;
      }
      __syncwarp();
      return true;
    }
    before += all;
  }
  return false;
}

// 256 rows of one kv head
struct Work {
  int h, q0, nq, k0, shift, window;
  int row0, tok0, tok1;  // first row, its token, one past the last token
  int t_lo, n;           // first key tile, their number (0: no row sees a key)
  bool two;              // the second tile has rows
  __device__ int tile(int j) const { return t_lo + n - 1 - j; }
  // does some row see only a part of tile j?
  __device__ bool partial(int j) const {
    const int a = tile(j) * kKeys;
    return a + kKeys - 1 > tok0 + shift || (window > 0 && a < tok1 + shift - window);
  }
};
__device__ bool find_work(const PromptAttn& p, volatile Place* place, int idx, Work& w) {
  int seq, tile;
  w.h = idx % p.n_kv_heads;
  if (!find_tile(p, place, idx / p.n_kv_heads, seq, tile)) return false;
  const Seq sq = prompt_seq(p, seq);
  w.q0 = sq.q0;
  w.nq = sq.nq;
  w.k0 = sq.k0;
  w.shift = sq.nk - sq.nq;
  w.window = p.window;
  w.row0 = tile * kBlockRows;
  w.tok0 = w.row0 / p.group;
  w.tok1 = min(sq.nq, w.tok0 + kBlockRows / p.group);
  const int hi = max(0, w.tok1 + w.shift), lo = p.window > 0 ? max(0, w.tok0 + w.shift - p.window + 1) : 0;
  w.t_lo = lo / kKeys;
  w.n = hi > 0 ? (hi + kKeys - 1) / kKeys - w.t_lo : 0;
  w.two = w.row0 + kRows < sq.nq * p.group;
  return true;
}

// A block's pieces of work: one of every round of gridDim.x, the rounds alternately from the front
// and from the back.  (The work is listed from the longest to the shortest: the
// block that got the longest piece of a round gets the shortest of the next.)
__device__ __forceinline__ bool next_work(const PromptAttn& p, volatile Place* place, int n_work, Work& w) {
  const int round = place->round;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) place->round = round + 1;
  const int64_t idx = (int64_t)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  return idx < n_work && find_work(p, place, (int)idx, w);
}

// The ring of K and V tiles, in the order K(0), V(0), K(1), V(1), ... of one piece of work
// after the other, as one of its readers walks it.  Every reader waits for every tile, so that none
// can fall or run a turn of the ring behind or ahead (a barrier only tells neighbouring phases
// apart).  A V has no signal of its own: a reader releases it with the K behind it, which for the last V of a
// piece of work is the next piece's first K.  That signal therefore has to come after the
// products that read the V, also from the thread of a tile that the next piece does not have.
template <int kStages>
struct Ring {
  int st = 0;
  uint32_t phase = 0;
  // waits for the next tile and returns its stage, -1 when it did not come
  __device__ __forceinline__ int next(uint64_t* full, volatile int* dead) {
    const int now = st;
    if (!wait_bar(&full[now], phase, dead)) return -1;
    if (++st == kStages) {
      st = 0;
      phase ^= 1;
    }
    return now;
  }
};

template <class El, int HD>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ Maps maps, const PromptAttn p, const int n_work) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t b_q[2], b_full[C::kStages], b_empty[C::kStages], b_clean[C::kStages], b_s[2], b_p[2],
      b_o[2], b_used[2], b_turn[2], b_drain[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_taken;
  __shared__ Place s_place[kPromptThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_q = smem;
  uint8_t* const s_kv = smem + 2 * C::kTileBytes;

  volatile Place* const place = &s_place[wid];
  if (lane == 0) place->round = place->c = place->before = 0;
  if (wid == 8) tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&b_q[t], 1);
      mbar_init(&b_s[t], 1);
      mbar_init(&b_p[t], 4);
      mbar_init(&b_o[t], 1);
      mbar_init(&b_used[t], 1);
      mbar_init(&b_turn[t], 1);
      mbar_init(&b_drain[t], 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 3);  // the readers: warps 8, 10 and 11
      mbar_init(&b_clean[i], 1);
    }
    s_dead = s_taken = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_shared();
  }
  if (tid >= kPromptThreads - 3) {
    const int m = kPromptThreads - 1 - tid;
    prefetch_tensormap(m == 0 ? &maps.q : m == 1 ? &maps.k : &maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // tensor memory: S (and P) of the two tiles, then O
  auto t_s = [&](int t) { return tmem + t * 128; };
  auto t_o = [&](int t) { return tmem + 256 + t * HD; };
  volatile int* const dead = &s_dead;
  Work w;

  if (wid >= 8) {
    set_max_regs_down<kOtherRegs>();
    if (wid == 9) {
      // ---- loads
      int i = 0, q_loads[2] = {0, 0};
      bool ok = true;
      // once the work before has its last scores: the next Q travels during that step's softmax
      auto load_q = [&](int t) {
        if (q_loads[t] > 0 && !wait_bar(&b_used[t], (q_loads[t] - 1) & 1, dead)) return false;
        ++q_loads[t];
        mbar_expect_tx(&b_q[t], C::kTileBytes);
        for (int x = 0; x < C::kBoxes; ++x)
          tma_load_4d(s_q + t * C::kTileBytes + x * kBoxBytes, &maps.q, x * 64, 0, w.h,
                      w.q0 + w.tok0 + t * (kRows / p.group), &b_q[t]);
        return true;
      };
      while (ok && !p.drop && next_work(p, place, n_work, w)) {
        if (lane == 0) {
          for (int e = 0; ok && e < 2 * w.n; ++e) {
            const int st = i % C::kStages;
            // the tile that the stage held, i - kStages, is used up; if it was a V, with the K
            // behind it.  (With an odd number of stages a stage holds a K every other time.)
            const int before = i - C::kStages, sig = before + (before & 1);
            constexpr int kTurn = C::kStages % 2 ? 2 * C::kStages : C::kStages;
            if (before >= 0 && !(ok = wait_bar(&b_empty[sig % C::kStages], (sig / kTurn) & 1, dead))) break;
            mbar_expect_tx(&b_full[st], C::kTileBytes);
            const CUtensorMap* const map = e & 1 ? &maps.v : &maps.k;
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(s_kv + st * C::kTileBytes + x * kBoxBytes, map, x * 64, w.h, w.k0 + w.tile(e >> 1) * kKeys,
                          &b_full[st]);
            ++i;
            if (e == 0) ok = load_q(0) && (!w.two || load_q(1));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0 && *dead) {  // nothing of this block may be on its way when it ends
        int never = 0;
        for (int t = 0; t < 2; ++t)
          if (q_loads[t] > 0) wait_bar(&b_q[t], (q_loads[t] - 1) & 1, &never);
        for (int k = max(0, i - C::kStages); k < i; ++k)
          wait_bar(&b_full[k % C::kStages], (k / C::kStages) & 1, &never);
      }
    } else if (wid == 8 || wid == 10) {
      // ---- products of one tile.  A round of waits and commits takes its thread some 600 cycles
      // beside the 1,024 of its products; with one thread for both tiles the tensor cores
      // idled meanwhile (3,400 cycles a step, 2,048 of them products).  The two threads take
      // turns: left to themselves both tiles fall into step, their products and then their
      // softmaxes at the same time.
      const int t = wid == 8 ? 0 : 1;
      const uint32_t i_s = idesc_f16(El::kBf16, p.scale_log2 < 0.f, false, kKeys);
      const uint32_t i_o = idesc_f16(El::kBf16, false, true, HD);
      const uint64_t d_q = sdesc_k_sw128(smem_u32(s_q)), d_k = sdesc_k_sw128(smem_u32(s_kv)),
                     d_v = sdesc_mn_sw128(smem_u32(s_kv), kBoxBytes);
      constexpr uint32_t kTile16 = C::kTileBytes >> 4;  // (descriptors count 16 bytes)
      constexpr int kTurnAt = HD / 16 - 1;
      const uint32_t ts = t_s(t), to = t_o(t);
      auto scores = [&](int st, bool turn) {  // S = Q K^T
        const uint64_t a = d_q + (uint32_t)t * kTile16, b = d_k + (uint32_t)st * kTile16;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = ((k / 4) * kBoxBytes + (k % 4) * 32) >> 4;
          // (the other thread needs some 150 cycles to notice; much earlier and its products delay
          // these: 1,388 us for 16,384 tokens here, 1,427 behind the last one, 1,438 halfway)
          if (k == kTurnAt && turn) mbar_arrive(&b_turn[1 - t], 1);
          mma_f16_ss(ts, a + off, b + off, i_s, k > 0);
        }
        tc_commit(&b_s[t]);
      };
      auto values = [&](int st, bool first) {  // O += P V
        const uint64_t b = d_v + (uint32_t)st * kTile16;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) mma_f16_ts(to, ts + k * 8, b + (k * 2048 >> 4), i_o, !first || k > 0);
      };
      Ring<C::kStages> ring;
      uint32_t clean_phase = 0;
      int steps = 0, loads = 0, turns = 0;  // of this tile's P and Q, and of the two threads, so far
      bool ok = true;
      Work ahead;
      for (bool more_work = next_work(p, place, n_work, ahead); ok && more_work;) {
        w = ahead;
        int k_st = -1;
        const bool mine = t == 0 || w.two;  // without a second tile its thread only signs the ring
        if (lane == 0 && w.n > 0) {
          k_st = ring.next(b_full, dead);
          ok = k_st >= 0 && (!mine || wait_bar(&b_q[t], loads++ & 1, dead));
          if (ok && mine) {
            tc_fence_after();
            scores(k_st, false);
            tc_commit(&b_empty[k_st]);
            if (w.n == 1) tc_commit(&b_used[t]);
          } else if (ok) {
            // (a commit, not an arrival: this thread's product of the last piece's last V, which this
            // releases too, may still be under way)
            tc_commit(&b_empty[k_st]);
          }
        }
        __syncwarp();
        // (looked up during the first softmax: behind the last product its loads wait for the
        // results' stores, 1,500 to 5,000 cycles)
        more_work = next_work(p, place, n_work, ahead);
        if (lane == 0 && w.n > 0) {
          for (int j = 0; ok && j < w.n; ++j) {
            const bool more = j + 1 < w.n;
            const int v_st = ring.next(b_full, dead);
            ok = v_st >= 0;
            if (!ok) break;
            if (w.partial(j)) {
              if (mine && !(ok = wait_bar(&b_clean[v_st], clean_phase >> v_st & 1, dead))) break;
              clean_phase ^= 1u << v_st;
            }
            if (more && !(ok = (k_st = ring.next(b_full, dead)) >= 0)) break;
            if (!mine) {
              if (more) mbar_arrive(&b_empty[k_st], 1);
              continue;
            }
            if (!(ok = wait_bar(&b_p[t], steps++ & 1, dead))) break;
            if (w.two) {
              if ((t == 1 || turns > 0) && !(ok = wait_bar(&b_turn[t], (t == 1 ? turns : turns - 1) & 1, dead))) break;
              ++turns;
            }
            tc_fence_after();
            values(v_st, j == 0);
            if (more) {
              scores(k_st, w.two);
              // V(j) and K(j + 1) are used up together: one signal, on K's stage.  (The last V's comes
              // with the next work's first K.)
              tc_commit(&b_empty[k_st]);
              if (j + 2 == w.n) tc_commit(&b_used[t]);
            } else {
              if (w.two) mbar_arrive(&b_turn[1 - t], 1);
              tc_commit(&b_o[t]);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0 && *dead) {  // no product may be under way when the block ends
        int never = 0;
        tc_commit(&b_drain[t]);
        wait_bar(&b_drain[t], 0, &never);
      }
    } else if (wid == 11) {
      // ---- finite check of the V tiles that some row sees in part
      constexpr uint32_t kE = El::kExponent, kLow = kE & (~kE + 1u);  // exponent field, its lowest bit
      Ring<C::kStages> ring;
      bool ok = true;
      while (ok && next_work(p, place, n_work, w)) {
        for (int e = 0; e < 2 * w.n; ++e) {
          const int st = ring.next(b_full, dead);
          if (!(ok = __all_sync(0xffffffffu, st >= 0))) break;
          if (e % 2 == 0) {
            if (lane == 0) mbar_arrive(&b_empty[st], 1);
            continue;
          }
          if (!w.partial(e >> 1)) continue;
          uint4* const v = reinterpret_cast<uint4*>(s_kv + st * C::kTileBytes);
          bool any = false;
          // (kBatch loads at a time: one by one, as the stores below them would keep them, 77,824 tokens on
          // a window of 128 keys took 595 us, and 501 so)
          constexpr int kBatch = 16;
          for (int c0 = lane; c0 < C::kTileBytes / 16; c0 += 32 * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) x[i] = v[c0 + 32 * i];
            // an exponent of all ones carries into the sign's place
            constexpr uint32_t m = kE * 0x10001u, a = kLow * 0x10001u;
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              bad |= ((x[i].x & m) + a) | ((x[i].y & m) + a) | ((x[i].z & m) + a) | ((x[i].w & m) + a);
            if (bad & 0x80008000u) {
              any = true;
              for (int i = 0; i < kBatch; ++i) {
                uint16_t* const el = reinterpret_cast<uint16_t*>(v + c0 + 32 * i);
                for (int q = 0; q < 8; ++q)
                  if ((el[q] & kE) == kE) el[q] = 0;
              }
            }
          }
          if (any) {
            s_taken = 1;  // (for all of the block's further work: its rows then look for themselves)
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_clean[st], 1);
        }
      }
    }
  } else {
    // ---- softmax: thread = row
    set_max_regs_up<kSoftmaxRegs>();
    const int t = wid >> 2;
    const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
    const uint32_t ts = t_s(t) + lanes, to = t_o(t) + lanes;
    // (a negative scale negates Q in the product; a scale of zero must still leave -inf x scale = -inf: the
    // smallest number does, and any score times it is less than 2^-20)
    const float scale = fmaxf(fabsf(p.scale_log2), __int_as_float(1));
    int steps = 0, works = 0;
    Work ahead;
    for (bool more = next_work(p, place, n_work, ahead); more;) {
      w = ahead;
      if (w.n > 0 && t == 1 && !w.two) {
        more = next_work(p, place, n_work, ahead);
        continue;
      }
      const int row = w.row0 + t * kRows + (wid & 3) * 32 + lane;
      const int tok = row / p.group, head = w.h * p.group + row % p.group;
      const int last = tok + w.shift;                                // the last key that the row sees
      const int first = w.window > 0 ? max(0, last - w.window + 1) : 0;  // and the first one
      uint16_t* const dst = p.out + (int64_t)(w.q0 + tok) * p.out_token + head * p.out_head;
      if (w.n == 0) {  // no row sees a key
        if (tok < w.nq)
          for (int c = 0; c < HD / 8; ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0u, 0u, 0u, 0u);
        more = next_work(p, place, n_work, ahead);
        continue;
      }
      float m = -INFINITY;
      uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      bool ok = !*dead;
      for (int j = 0; ok && j < w.n; ++j) {
        ok = __all_sync(0xffffffffu, wait_bar(&b_s[t], steps++ & 1, dead));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s[c]);
        tmem_ld_wait();
        if (w.partial(j)) {
          const int a = first - w.tile(j) * kKeys, b = last - w.tile(j) * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = bits_upto(b - c * 32) & ~bits_upto(a - 1 - c * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[c][i] = see >> i & 1 ? s[c][i] : 0xFF800000u;
          }
        }
        // P from the scores with the maximum so far, and the tile's own maximum on the side
        float mx;
        uint64_t sum[2];
        auto weights = [&]() {
          const float neg = m == -INFINITY ? 0.f : kTop<El> - m * scale;
          const uint64_t sc2 = pair(scale, scale), neg2 = pair(neg, neg);
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          sum[0] = sum[1] = pair(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float s0 = __uint_as_float(s[c][2 * i]), s1 = __uint_as_float(s[c][2 * i + 1]);
              float e0, e1;
              unpair(fma2(pair(s0, s1), sc2, neg2), e0, e1);
              x[i & 3] = max3(x[i & 3], s0, s1);
              e0 = exp2_fast(e0);
              e1 = exp2_fast(e1);
              sum[i & 1] = add2(sum[i & 1], pair(e0, e1));
              // Rounded to the 16-bit type for the product with V; the sum keeps 32 bits.  (The rest as a
              // second term, a second product: relative L2 error 2.1e-3 -> 1.6e-3, what the
              // result's own rounding leaves, fp16 2.6e-4 -> 2.0e-4, but 16,384 tokens 1.39 -> 2.39 ms.)
              pk[i] = El::pack(e0, e1);
            }
            tmem_st16(ts + c * 16, pk);
          }
          mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        };
        // the first tile that a row sees (nothing of the row is in O and the sum yet)
        if (__any_sync(0xffffffffu, m == -INFINITY)) {
          float own = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2) own = max3(own, __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
          if (m == -INFINITY) m = own;
        }
        weights();
        const bool grow = (mx - m) * scale > kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? exp2_fast((m - mx) * scale) : 1.f;
          if (grow) m = mx;
          const uint64_t ff = pair(f, f), zero = pair(0.f, 0.f);
          l2[0] = fma2(l2[0], ff, zero);
          l2[1] = fma2(l2[1], ff, zero);
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + c * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to + c * 16, o);
          }
          weights();
        }
        l2[0] = add2(l2[0], sum[0]);
        l2[1] = add2(l2[1], sum[1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_p[t], 1);
      }
      more = next_work(p, place, n_work, ahead);  // (looked up while the last product runs)
      ok = ok && __all_sync(0xffffffffu, wait_bar(&b_o[t], works++ & 1, dead));
      tc_fence_after();
      float l0, l1;
      unpair(add2(l2[0], l2[1]), l0, l1);
      // no key seen: zeros; a wait that ran out: NaN
      const float inv = !ok ? NAN : last < 0 ? 0.f : 1.f / (l0 + l1);
      const bool taken = *(volatile int*)&s_taken != 0;
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
              const uint16_t* const v = p.v + (int64_t)(w.k0 + key) * p.v_token + w.h * p.v_head + c * 32;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((v[i] & El::kExponent) == El::kExponent) f[i] += El::value(v[i]);
            }
          }
        }
        if (tok < w.nq) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = El::pack(f[2 * i], f[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            uint16_t* const d = dst + c * 32 + 2 * i;
            if (p.out_32) {
              st_global_32(d, &h[i]);
            } else {
              reinterpret_cast<uint4*>(d)[0] = make_uint4(h[i], h[i + 1], h[i + 2], h[i + 3]);
              reinterpret_cast<uint4*>(d)[1] = make_uint4(h[i + 4], h[i + 5], h[i + 6], h[i + 7]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_dead && p.status) atomicCAS(p.status, 0, MSM_ERR_DEVICE_TIMEOUT);
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
cudaError_t launch(const PromptAttn& p, int sms, cudaStream_t s) {
  const int64_t works = prompt_attn_works(p.n_q, p.n_seqs, p.n_kv_heads, p.group);
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
  prompt_kernel<El, HD><<<(unsigned)std::min<int64_t>(works, sms), kPromptThreads, Cfg<HD>::kSmem, s>>>(maps, p, (int)works);
  return cudaGetLastError();
}

}  // namespace

int64_t prompt_attn_works(int n_q, int n_seqs, int n_kv_heads, int group) {
  return (((int64_t)n_q * group + kBlockRows - 1) / kBlockRows + n_seqs) * n_kv_heads;
}

cudaError_t launch_prompt_attn(const PromptAttn& p, int dtype, int head_dim, int sms, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, sms, s) : launch<Bf16, 128>(p, sms, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, sms, s) : launch<Fp16, 128>(p, sms, s);
}

}  // namespace msm
