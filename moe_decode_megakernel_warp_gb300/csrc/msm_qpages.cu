// msm_qpages.cu — storing new K/V rows in a paged cache of 8 bits (msm_qpages_write):
//   value = e4m3 code x scale, one 32-bit scale for the rows of a block (block_rows rows of one page and
//   head), K and V apart.
//
// With amax the largest finite magnitude of a block's new rows, the least power of two s with
// amax <= 448 s is what they need.  A block without older rows takes it; one with older rows keeps the
// larger of it and what it has, and where that grows the older codes are multiplied by old / new and
// rounded again.  Between powers of two this loses nothing but bits of values below 2^-6 of the scale
// (a floating-point code has the same 4 bits at every size), so rows that come one at a time end up as
// rows that come together do, up to those.
//
// Bound by memory for prompts (2 bytes read, 1 written per element) and by latency for a step's few
// tokens.  A unit of threads, one warp or a block of eight warps, takes the blocks of rows that begin
// among `group` tokens, for one head of K or V: a unit's loads are on their way before it knows the
// largest element, and stay in registers until they are stored (a second read where a block has more
// rows than that).  No two units meet in a block of rows, so no atomics.
#include "msm_attn.cuh"
#include "msm_paged.h"

namespace msm {
namespace {

constexpr int kHeld = 8;      // 16-byte vectors in registers per lane
constexpr int kManyWarps = 8;
constexpr int kFewThreads = 128;

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

// kWarps warps work on a unit together; a block holds one such unit, or four of a warp
template <class El, int HD, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? kFewThreads : kWarps * 32) qwrite_kernel(const QPagesWrite p) {
  constexpr int kVecs = HD / 8;             // 16-byte vectors of a new row
  constexpr int kRows = 32 / kVecs * kWarps;  // new rows of one step
  constexpr int kUnits = kWarps == 1 ? kFewThreads / 32 : 1;
  __shared__ uint32_t s_max[2][kWarps];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int w = kWarps == 1 ? 0 : wid;
  const int c = lane % kVecs, sub = w * (32 / kVecs) + lane / kVecs;
  const int limit = min(p.n_tokens, max(p.starts[p.m.n_seqs], 0));
  const int groups = (limit - 1) / p.group + 1;
  if (limit == 0) return;
  const bool stop = stopped(p.m.status);
  if (stop) return;
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
  for (int64_t unit = (int64_t)blockIdx.x * kUnits + (kWarps == 1 ? wid : 0); unit < (int64_t)groups * 2 * p.n_kv_heads;
       unit += (int64_t)gridDim.x * kUnits) {
    const int head = (int)(unit % p.n_kv_heads), is_v = (int)(unit / p.n_kv_heads & 1);
    const int64_t t_first = unit / p.n_kv_heads / 2 * p.group;
    const int t_end = (int)min((int64_t)limit, t_first + p.group);
    const uint16_t* const src = (is_v ? p.v : p.k) + head * (is_v ? p.v_head : p.k_head);
    const int64_t token = is_v ? p.v_token : p.k_token;
    uint8_t* const pool = is_v ? p.pool_v : p.pool_k;
    float* const scales = is_v ? p.v_scales : p.k_scales;
    auto load = [&](int t) { return __ldcs(reinterpret_cast<const uint4*>(src + t * token) + c); };
    for (int t = (int)t_first; t < t_end;) {
      // most units: the rows of one block, from the group's first token on (their loads do not wait for the search)
      uint4 x[kHeld];
      const int t_loaded = t;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int r = i * kRows + sub;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.group && r < limit - t) x[i] = load(t + r);
      }
      // the last sequence that starts at or before the token, 32 probes at a time
      int lo = 0, hi = p.m.n_seqs;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const uint32_t le = __ballot_sync(0xffffffffu, i < hi && p.starts[i] <= t);
        lo += le ? (31 - __clz(le)) * step : 0;
        hi = min(hi, lo + step);
      }
      const int first = p.starts[lo], end = p.starts[lo + 1];
      bool bad = t < first || t >= end;
      const int64_t pos = (int64_t)p.m.lens[lo] - end + t;
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
      const int in_page = (int)pos % p.m.page_rows, block = in_page / p.block_rows, row0 = block * p.block_rows;
      const int older = in_page - row0, left = min(p.block_rows - older, p.m.page_rows - in_page);
      const int n = min(left, next - t);
      if (older > 0 && t != first) {  // another unit's, which has the block's first new row
        t += n;
        continue;
      }
      const int pg = p.m.table[(size_t)lo * p.m.max_pages + (int)pos / p.m.page_rows];
      if (pg < 0 || pg >= p.m.n_pages || p.m.refs[pg] != 1) {
        if (lane == 0 && w == 0) latch(p.m.status, MSM_ERR_INVALID_ARG, kCallWrite);
        t += n;
        continue;
      }
      const int64_t at = (int64_t)pg * p.n_kv_heads + head;
      float* const scale = scales + at * p.page_blocks + block;
      uint8_t* const rows = pool + (at * p.m.page_rows + row0) * HD;
      const float old = older > 0 ? *scale : 0.f;

      // what is held in registers begins at t_loaded = t (a group begins, or the loop came around)
      auto step_of = [&](int i0, uint4 (&y)[kHeld]) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int r = i0 + i * kRows + sub;
          y[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < n) y[i] = load(t_loaded + r);
        }
      };
      uint32_t most = 0;
      auto add = [&](const uint4 (&y)[kHeld], int i0, bool finite) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (i0 + i * kRows + sub < n) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t v = (&y[i].x)[q];
              most = max_abs2<El>(most, finite ? finite2<El>(v) : v);
            }
          }
      };
      // (rows behind the group's end belong to it as well)
      constexpr int kIn = kHeld * kRows;
      if (n > p.group) step_of(0, x);
      add(x, 0, false);
      for (int i0 = kIn; i0 < n; i0 += kIn) {
        uint4 y[kHeld];
        step_of(i0, y);
        add(y, i0, false);
      }
      uint32_t top = largest(most);
      if (top >= El::kExponent) {  // an infinite element: the largest finite one decides
        most = 0;
        add(x, 0, true);
        for (int i0 = kIn; i0 < n; i0 += kIn) {
          uint4 y[kHeld];
          step_of(i0, y);
          add(y, i0, true);
        }
        top = largest(most);
      }
      const float now = fmaxf(old, scale_for(El::value((uint16_t)top)));
      if (now != old) {
        // the older rows on the new scale
        const float ratio = old / now;
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
      const float inverse = now > 0.f ? 1.f / now : 0.f;
      auto store = [&](const uint4 (&y)[kHeld], int i0) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int r = i0 + i * kRows + sub;
          if (r < n) {
            float f[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = El::value((uint16_t)((&y[i].x)[q >> 1] >> (16 * (q & 1)))) * inverse;
            uint2 o;
            o.x = pack_e4m3(f[0], f[1], f[2], f[3]);
            o.y = pack_e4m3(f[4], f[5], f[6], f[7]);
            reinterpret_cast<uint2*>(rows + (int64_t)(older + r) * HD)[c] = o;
          }
        }
      };
      store(x, 0);
      for (int i0 = kIn; i0 < n; i0 += kIn) {
        uint4 y[kHeld];
        step_of(i0, y);
        store(y, i0);
      }
      // (every thread has read the old one: there was a barrier since)
      if (lane == 0 && w == 0) *scale = now;
      t += n;
    }
  }
}

template <class El, int HD>
cudaError_t launch(const QPagesWrite& p, cudaStream_t s) {
  const int64_t units = ((int64_t)(p.n_tokens - 1) / p.group + 1) * 2 * p.n_kv_heads;
  const int64_t most = 1 << 30;
  // Eight warps where a block of rows is more than a warp holds in registers: also a step's few tokens may have
  // to multiply all of its older rows.
  if (p.block_rows > kHeld * (32 / (HD / 8)))
    qwrite_kernel<El, HD, kManyWarps><<<(unsigned)(units < most ? units : most), kManyWarps * 32, 0, s>>>(p);
  else
    qwrite_kernel<El, HD, 1><<<(unsigned)((units - 1) / (kFewThreads / 32) + 1 < most ? (units - 1) / (kFewThreads / 32) + 1 : most),
                               kFewThreads, 0, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_qpages_write(const QPagesWrite& p, int dtype, int head_dim, cudaStream_t s) {
  if (dtype == MSM_BF16) return head_dim == 64 ? launch<Bf16, 64>(p, s) : launch<Bf16, 128>(p, s);
  return head_dim == 64 ? launch<Fp16, 64>(p, s) : launch<Fp16, 128>(p, s);
}

}  // namespace msm
