// msm_qpages.cu — storing new K/V rows in a paged cache of 8 bits (msm_qpages_write):
//   value = e4m3 code x scale, one 32-bit scale for the rows of a block (block_rows rows of one page and
//   head), K and V apart.
//
// With amax the largest finite magnitude of a block's new rows, the least power of two s with
// amax <= 448 s is what they need.  A block without older rows takes it; one with older rows keeps the
// larger of it and what it has, and where that grows the older codes are multiplied by old / new and
// rounded again.  New elements are divided by the scale, exactly: a power of two has an exact reciprocal, and
// with other scales, which only a cache from elsewhere has, the remainder decides (quotient).  Between powers
// of two this loses nothing but bits of values below 2^-6 of the scale (a floating-point code has the same 4
// bits at every size), so rows that come one at a time end up as rows that come together do, up to those.
//
// Bound by memory for prompts (2 bytes read, 1 written per element) and by latency for a step's few
// tokens.  A unit, one to eight warps, takes the blocks of rows that begin among `group` tokens, K and V of
// one head.  The rows' loads are on their way while the page is looked up, and stay in registers from the
// search for the largest element until they are stored (a second read where a block has more rows than that).
// No two units meet in a block of rows, so no atomics.
//
// On one GB300 50,000 tokens of 8 heads of 128 in blocks of 16 rows take 52 - 54 us on the GPU (5,700 - 5,900 GB/s;
// the resize in front of them 8, of which its launch hides some), in blocks of 64 rows 54 - 57, of 256 rows
// 126.  How many warps share a unit follows the tokens per slot of the table, so a prompt in a table of many
// empty slots is slow in long blocks: 4,096 tokens among 512 slots in blocks of 256 rows 102 us.
// K and V apart, a warp each: 60 us (the way from a token to its page is a chain of loads, which the two then
// share); rows loaded before it is known which of the group's tokens begins a block: 72.
#include "msm_attn.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kHeld = 8;      // 16-byte vectors in registers per lane

// two fp32 values as e4m3, to nearest even, infinities to the largest value
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t x, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
  f[0] = Fp16::value((uint16_t)lo);
  f[1] = Fp16::value((uint16_t)(lo >> 16));
  f[2] = Fp16::value((uint16_t)hi);
  f[3] = Fp16::value((uint16_t)(hi >> 16));
}

// x / s for the rounding to a code, with `inverse` the rounded 1 / s: a number on the same side of every border between two
// codes as the exact quotient, or on it with that.  Such a border has at most 5 bits.  The product rounded to 12 bits is either a border
// or has none between itself and the exact quotient (less than a step of 12 bits away), and which side of it that lies on
// is the sign of x - t s, which one operation gives.  (s from 2^-60 on, so that it does not vanish.)
__device__ __forceinline__ float quotient(float x, float s, float inverse) {
  const float q = x * inverse;
  const uint32_t t = (__float_as_uint(q) + 0x800u) & 0xFFFFF000u;
  const float rest = fmaf(-__uint_as_float(t), s, x);
  const uint32_t beside = (t ^ __float_as_uint(rest)) >> 31 ? t - 1 : t + 1;
  return rest == 0.f ? __uint_as_float(t) : fabsf(rest) > 0.f ? __uint_as_float(beside) : q;  // (q: an infinity, NaN)
}

// four 16-bit elements
template <class El>
__device__ __forceinline__ void four(uint32_t x, uint32_t y, float (&f)[4]) {
  if constexpr (El::kBf16) {
    f[0] = __uint_as_float(x << 16), f[1] = __uint_as_float(x & 0xFFFF0000u);
    f[2] = __uint_as_float(y << 16), f[3] = __uint_as_float(y & 0xFFFF0000u);
  } else {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x)), q = __half22float2(*reinterpret_cast<const __half2*>(&y));
    f[0] = p.x, f[1] = p.y, f[2] = q.x, f[3] = q.y;
  }
}
// times s
template <class El>
__device__ __forceinline__ uint32_t scaled_e4m3(uint32_t x, uint32_t y, float s) {
  float f[4];
  four<El>(x, y, f);
  return pack_e4m3(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
}

// the least power of two that amax / 448 does not exceed, at least 2^-126; 0 for 0
__device__ __forceinline__ float scale_for(float amax) {
  if (amax < 0x1p-118f) return amax > 0.f ? 0x1p-126f : 0.f;
  const uint32_t b = __float_as_uint(amax);  // amax = m 2^e; 448 = 1.75 x 2^8
  const uint32_t e = (b >> 23) - ((b & 0x7FFFFFu) <= 0x600000u ? 8u : 7u);
  return __uint_as_float(e << 23);
}

// largest magnitudes of two elements each
template <class El>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t x) {
  x &= 0x7FFF7FFFu;
  uint32_t r;
  if (El::kBf16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(x));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(x));
  return r;
}
template <class El>
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  if ((x & El::kExponent) == El::kExponent) x &= 0xFFFF0000u;
  if ((x >> 16 & El::kExponent) == El::kExponent) x &= 0xFFFFu;
  return x;
}

// blockIdx.x: the group of tokens; blockIdx.y: the head, which kWarps = 4 or 8 warps take together, or four heads of
// a warp each.  kLong: a block of rows may have more new rows than registers hold (the code for them costs the others
// registers: 50,000 tokens into blocks of 16 rows 56 us without it, 79 with it).
constexpr int threads(int warps) { return warps == 1 ? 128 : 32 * warps; }
template <class El, int HD, int kWarps, bool kLong>
__global__ void __launch_bounds__(threads(kWarps), 512 / threads(kWarps))
    qwrite_kernel(const QPagesWrite p) {
  constexpr int kVecs = HD / 8;               // 16-byte vectors of a new row
  constexpr int kRows = 32 / kVecs * kWarps;  // new rows of one step
  constexpr int kIn = kHeld * kRows;          // and of those that registers hold (more are read twice, kMore steps
  constexpr int kMore = 2;                    // at a time)
  __shared__ uint32_t s_max[2][kWarps];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int w = kWarps == 1 ? 0 : wid;
  const int c = lane % kVecs, sub = w * (32 / kVecs) + lane / kVecs;
  pdl_wait();
  // (up to 31 sequences: all of their starts and lengths at once, one wait instead of four in a row)
  const bool few = p.m.n_seqs < 32;
  const int my_start = few ? p.starts[min(lane, p.m.n_seqs)] : 0, my_len = few ? p.m.lens[min(lane, p.m.n_seqs - 1)] : 0;
  const int limit = min(p.n_tokens, max(few ? __shfl_sync(0xffffffffu, my_start, p.m.n_seqs) : p.starts[p.m.n_seqs], 0));
  const int64_t t_first = (int64_t)blockIdx.x * p.group;
  const int head = kWarps == 1 ? (int)blockIdx.y * 4 + wid : (int)blockIdx.y;
  if (t_first >= limit || head >= p.n_kv_heads || stopped(p.m.status)) return;
  const int64_t cap = (int64_t)p.m.max_pages * p.m.page_rows;
  int flip = 0;
  // the largest of all the unit's lanes' elements (two in each)
  auto largest = [&](uint32_t x) -> uint32_t {
    uint32_t m = __reduce_max_sync(0xffffffffu, max(x & 0xFFFFu, x >> 16));
    if constexpr (kWarps > 1) {
      if (lane == 0) s_max[flip][w] = m;
      __syncthreads();
      m = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) m = max(m, s_max[flip][i]);
      flip ^= 1;  // (the next call writes to the other half, so that one barrier is enough)
    }
    return m;
  };
  const int t_end = (int)min((int64_t)limit, t_first + p.group);
  for (int t = (int)t_first; t < t_end;) {
    // the last sequence that starts at or before the token, 32 probes at a time
    int lo = 0, first, end, len;
    if (few) {
      const uint32_t le = __ballot_sync(0xffffffffu, lane < p.m.n_seqs && my_start <= t);
      lo = le ? 31 - __clz(le) : 0;
      first = __shfl_sync(0xffffffffu, my_start, lo);
      end = __shfl_sync(0xffffffffu, my_start, lo + 1);
      len = __shfl_sync(0xffffffffu, my_len, lo);
    } else {
      for (int hi = p.m.n_seqs; hi - lo > 1;) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const uint32_t le = __ballot_sync(0xffffffffu, i < hi && p.starts[i] <= t);
        lo += le ? (31 - __clz(le)) * step : 0;
        hi = min(hi, lo + step);
      }
      first = p.starts[lo];
      end = p.starts[lo + 1];
      len = p.m.lens[lo];
    }
    bool bad = t < first || t >= end;
    const int64_t pos = (int64_t)len - end + t;
    int next = bad ? t + 1 : min(end, limit);
    if (!bad && pos < 0) {  // tokens in front of the sequence's first row
      bad = true;
      next = (int)min((int64_t)next, t - pos);
    }
    bad |= pos >= cap;
    if (bad) {
      if (lane == 0 && w == 0) latch(p.m.status, MSM_ERR_INVALID_ARG, kCallWrite);
      t = next;
      continue;
    }
    // the block of rows that holds the token's, and how many of the tokens go there
    const int page = (int)p.by_page.of((uint32_t)pos), in_page = (int)pos - page * p.m.page_rows;
    const int block = (int)p.by_block.of((uint32_t)in_page), row0 = block * p.block_rows;
    const int older = in_page - row0, left = min(p.block_rows - older, p.m.page_rows - in_page);
    const int n = min(left, next - t);
    if (older > 0 && t != first) {  // another unit's, which has the block's first new row
      t += n;
      continue;
    }
    // rows i0 + i kRows + sub of K or V (what is behind the n-th stays as it was)
    auto load = [&](bool is_v, int i0, auto& y) {
      const int64_t token = is_v ? p.v_token : p.k_token;
      const uint16_t* const from = (is_v ? p.v + head * p.v_head : p.k + head * p.k_head) + (t + i0 + sub) * token + c * 8;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(y) / sizeof(y[0])); ++i)
        if (i0 + i * kRows + sub < n) y[i] = __ldcs(reinterpret_cast<const uint4*>(from + i * kRows * token));
    };
    uint4 x[2][kHeld];  // K, V (these travel while the page is looked up)
#pragma unroll
    for (int side = 0; side < 2; ++side) load(side != 0, 0, x[side]);
    const int pg = p.m.table[(size_t)lo * p.m.max_pages + page];
    if (pg < 0 || pg >= p.m.n_pages || p.m.refs[pg] != 1) {
      if (lane == 0 && w == 0) latch(p.m.status, MSM_ERR_INVALID_ARG, kCallWrite);
      t += n;
      continue;
    }
    const int64_t at = (int64_t)pg * p.n_kv_heads + head;
    float old[2];
#pragma unroll
    for (int side = 0; side < 2; ++side)
      old[side] = older > 0 ? (side ? p.v_scales : p.k_scales)[at * p.page_blocks + block] : 0.f;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const bool is_v = side != 0;
      uint8_t* const rows = (is_v ? p.pool_v : p.pool_k) + (at * p.m.page_rows + row0) * HD;
      uint32_t most = 0;
      auto add = [&](const auto& y, int i0, bool finite) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(y) / sizeof(y[0])); ++i)
          if (i0 + i * kRows + sub < n) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t v = (&y[i].x)[q];
              most = max_abs2<El>(most, finite ? finite2<El>(v) : v);
            }
          }
      };
      auto add_all = [&](bool finite) {
        add(x[side], 0, finite);
        if constexpr (kLong) {
#pragma unroll 1
          for (int i0 = kIn; i0 < n; i0 += kMore * kRows) {
            uint4 y[kMore];
            load(is_v, i0, y);
            add(y, i0, finite);
          }
        }
      };
      add_all(false);
      uint32_t top = largest(most);
      if (top >= El::kExponent) {  // an infinite element: the largest finite one decides
        most = 0;
        add_all(true);
        top = largest(most);
      }
      const float now = fmaxf(old[side], scale_for(El::value((uint16_t)top)));
      if (now != old[side]) {
        // the older rows on the new scale
        const float ratio = old[side] / now;
        constexpr int kOld = HD / 16, kOldRows = 32 / kOld * kWarps;  // 16-byte vectors of a row, rows of one step
        for (int r0 = 0; r0 < older; r0 += 4 * kOldRows) {
          uint4 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + i * kOldRows + w * (32 / kOld) + lane / kOld;
            if (r < older) y[i] = reinterpret_cast<const uint4*>(rows + (int64_t)r * HD)[lane % kOld];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + i * kOldRows + w * (32 / kOld) + lane / kOld;
            if (r < older) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float f[4];
                unpack_e4m3((&y[i].x)[q], f);
                (&y[i].x)[q] = pack_e4m3(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
              }
              reinterpret_cast<uint4*>(rows + (int64_t)r * HD)[lane % kOld] = y[i];
            }
          }
        }
      }
      // New elements over the scale.  A power of two from 2^-126 on has an exact reciprocal, whose bits are those of 2^127 less its
      // own.  With a scale below that, 0 among them, the only finite new element is 0: 0 stays 0, and infinities become +-448.
      const uint32_t bits = __float_as_uint(now);
      uint8_t* const to = rows + (int64_t)(older + sub) * HD + c * 8;
      if (bits <= 1u << 23 || (bits << 9 == 0 && bits < 254u << 23)) {
        const float inverse = bits >= 1u << 23 ? __uint_as_float((254u << 23) - bits) : 1.f;
        auto store = [&](const auto& y, int i0) {
#pragma unroll
          for (int i = 0; i < (int)(sizeof(y) / sizeof(y[0])); ++i)
            if (i0 + i * kRows + sub < n) {
              uint2 o;
              o.x = scaled_e4m3<El>(y[i].x, y[i].y, inverse);
              o.y = scaled_e4m3<El>(y[i].z, y[i].w, inverse);
              *reinterpret_cast<uint2*>(to + (int64_t)i0 * HD + i * kRows * HD) = o;
            }
        };
        store(x[side], 0);
        if constexpr (kLong) {
#pragma unroll 1
          for (int i0 = kIn; i0 < n; i0 += kMore * kRows) {
            uint4 y[kMore];
            load(is_v, i0, y);
            store(y, i0);
          }
        }
      } else {
        // Any other scale is one that the block came with, and divides.  (A row at a time, read again, so that this takes few
        // registers of the way above: 50,000 tokens in blocks of 16 rows 53.6 -> 54.3 us, of 64 56.3 -> 57.1, of 256 119 -> 126.
        // As a function, or behind all stores, 3 to 55 us.)
        const float up = now < 0x1p-60f ? 0x1p64f : 1.f, by = now * up, inverse = 1.f / by;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kRows) {
          uint4 y[1];
          load(is_v, i0, y);
#pragma unroll 1
          for (int q = 0; q < 2 && i0 + sub < n; ++q) {
            float f[4];
            four<El>(q ? y[0].z : y[0].x, q ? y[0].w : y[0].y, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = quotient(f[i] * up, by, inverse);
            *reinterpret_cast<uint32_t*>(to + (int64_t)i0 * HD + 4 * q) = pack_e4m3(f[0], f[1], f[2], f[3]);
          }
        }
      }
      // (every thread has read the old one: there was a barrier since)
      if (lane == 0 && w == 0) (is_v ? p.v_scales : p.k_scales)[at * p.page_blocks + block] = now;
    }
    t += n;
  }
}

template <class El, int HD, int kWarps>
cudaError_t launch_of(const QPagesWrite& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.n_tokens - 1) / p.group + 1), kWarps == 1 ? (p.n_kv_heads - 1) / 4 + 1 : p.n_kv_heads);
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads(kWarps));
  lc.stream = s;
  cudaLaunchAttribute attr[1];  // started while the launch in front of it (the copies of a resize) ends
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return p.block_rows > kHeld * (32 / (HD / 8)) * kWarps ? cudaLaunchKernelEx(&lc, qwrite_kernel<El, HD, kWarps, true>, p)
                                                         : cudaLaunchKernelEx(&lc, qwrite_kernel<El, HD, kWarps, false>, p);
}
template <class El, int HD>
cudaError_t launch(const QPagesWrite& p, cudaStream_t s) {
  // as many warps as the tokens that come together to a block of rows keep busy
  constexpr int kWarpRows = kHeld * (32 / (HD / 8));
  if (p.group <= kWarpRows) return launch_of<El, HD, 1>(p, s);
  return p.group <= 4 * kWarpRows ? launch_of<El, HD, 4>(p, s) : launch_of<El, HD, 8>(p, s);
}
}  // namespace

cudaError_t launch_qpages_write(const QPagesWrite& p, int dtype, int head_dim, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, s) : launch<Bf16, 128>(p, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, s) : launch<Fp16, 128>(p, s);
}

}  // namespace msm
