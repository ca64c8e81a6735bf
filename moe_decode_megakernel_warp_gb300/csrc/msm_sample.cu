// msm_sample.cu — drawing tokens from logits (msm_sample): temperature, top-k, top-p, min-p, and one
// given random number per row.
//
// With x the logits of a row, M their maximum and w_i = exp((x_i - M) / T), in the order "larger logit
// first, lower index first among equals":
//   top-k keeps the first k; top-p, of these, the shortest beginning whose weights reach top_p of theirs;
//   min-p those with w >= min_p.  All three keep a beginning of the order.
//   The token is the lowest index whose weights, summed over the kept ones in the order of the index,
//   exceed random x their sum.
//
// Weights are whole multiples of 2^-42 (of the largest weight), so their sums are exact in 64 bits whatever
// their order: which token is drawn depends on no thread's timing, and the sums say the same as the
// definition in 64-bit floating point but for the weights' own rounding.  That is two roundings of a number of
// 1/2 .. 1 to 2^-31, together 1.1 x 2^-30 of the weight, and one to 2^-42, which is 2^-43 of the largest weight:
// below 2^-13 of the largest the second counts (a weight of 2^-38 keeps five bits).  A sum is off by at most
// 1.1 x 2^-30 of itself and 2^-43 for each of its weights.  That matters: a row's 100,000 borders between tokens
// lie so close that weights of 32-bit floating point draw another token in one of some thousand rows.
// w = 2^-t, t = (M - x) log2(e) / T as two floats: t = k + j / 1024 + r, a table of 1,024 entries for j, a
// polynomial of third degree for r, two logits per instruction.
//
// A row belongs to one cluster of up to eight blocks, each with a slice of it in shared memory, so the
// logits are read once.  The order's border is found without sorting the row: a histogram over 1,024
// classes of t below 16 (counts and, where top-p needs them, weights), of which only the class that holds the
// border goes on: gathered and sorted by the cluster's first block when it is small (top-k: with all classes
// in front of it), else divided into 1,024 finer classes, down to single values, whose equals are told apart
// by index.  Between the steps the blocks exchange sums through distributed shared memory.
//
// Bound by instructions and by the chain of steps, not by memory (the logits of 500 rows are 7 us of DRAM): a weight is
// some 35 instructions, and top-p without top-k needs every logit's, those of the kept ones a second time for the draw; and
// the other blocks of a cluster wait at barriers (the largest stall) while the first one merges, searches and sorts.
// Measured on one GB300: one row of 32,003 fp32 logits, top-k 50 and top-p 12.5 us (some 8 us of steps, each 0.5 to 1.5 us:
// cluster barriers, reads of other blocks' memory, the sort of the list); 64 rows of 131,072 with settings of their
// own 60 us; 500 rows of 50,021 bf16 logits, top-p alone 159 us (ALU 48 %, issue slots 55 %; the histogram takes two
// fifths of a block's time, the sums for the draw a fifth, gathering the border's class an eighth).  256 threads a
// block, four blocks per SM: a tenth slower; counts and weights together where top-k is given 78 us where counts alone took 64 (64 rows); the rows behind
// the last full round of clusters in a launch of their own with more blocks each: 174 us where one launch takes 159.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

#include "msm_attn.cuh"
#include "msm_sample.h"

namespace cg = cooperative_groups;

namespace msm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 1024 / kThreads;
constexpr int kBins = 1024;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kList = kThreads;       // candidates that are sorted
constexpr int kSegs = 128;            // segments of a slice, in the order of the index
constexpr int kMaxCluster = 8;
constexpr int kBits = 42;             // weights are multiples of 2^-42 ...
constexpr uint64_t kOne = 0x7FFFFFFFull << (kBits - 31);  // ... of this one, the largest logit's (2^-31 short of 1)
constexpr uint32_t kLowestKey = 0x00800000u;  // of the lowest finite value

// 2^(-i / 32) in units of 2^-63 and 2^(-i / 1024) in units of 2^-64 (its first one a unit short of 1)
__constant__ uint64_t c_coarse[32] = {
    0x8000000000000000ull, 0x7d41d96db915019dull, 0x7a92be8a92436616ull, 0x77f25ccdee6d7ae6ull,
    0x75606373ee921c97ull, 0x72dc8373be41a454ull, 0x70666f76154a7089ull, 0x6dfddbcbed791babull,
    0x6ba27e656b4eb57aull, 0x69540ec8f895722dull, 0x6712460a8fc24072ull, 0x64dcdec3371793d1ull,
    0x62b39508aa836d6full, 0x6096266533384a2bull, 0x5e8451cfac061b5full, 0x5c7dd7a3b17dcf75ull,
    0x5a827999fcef3242ull, 0x5891fac0e95612c8ull, 0x56ac1f752150a563ull, 0x54d0ad5a753e077cull,
    0x52ff6b54d8a89c75ull, 0x513821818624b40cull, 0x4f7a993048d088d7ull, 0x4dc69cdceaa72a9cull,
    0x4c1bf828c6dc54b8ull, 0x4a7a77d47f7b84b1ull, 0x48e1e9b9d588e19bull, 0x47521cc5a2e6a9e0ull,
    0x45cae0f1f545eb73ull, 0x444c0740496d4294ull, 0x42d561b3e6243d8aull, 0x4166c34c5615d0ecull};
// (in global memory: a warp reads all 32 of them at once)
__device__ const uint64_t c_fine[32] = {
    0xffffffffffffffffull, 0xffd3a751c0f7e10cull, 0xffa756521c8daed2ull, 0xff7b0cffbe159675ull,
    0xff4ecb59511ec8a5ull, 0xff22915d81736f63ull, 0xfef65f0afb18a3caull, 0xfeca34606a4e63dcull,
    0xfe9e115c7b8f884cull, 0xfe71f5fddb91ba4bull, 0xfe45e2433745695dull, 0xfe19d62b3bd5c123ull,
    0xfdedd1b496a89f35ull, 0xfdc1d4ddf55e88f3ull, 0xfd95dfa605d2a15eull, 0xfd69f20b761a9ef0ull,
    0xfd3e0c0cf486c175ull, 0xfd122da92fa1c7e8ull, 0xfce656ded630e654ull, 0xfcba87ac9733bbafull,
    0xfc8ec01121e447bbull, 0xfc63000b25b6e0f0ull, 0xfc374799525a2a57ull, 0xfc0b96ba57b7097bull,
    0xfbdfed6ce5f09c49ull, 0xfbb44bafad642efdull, 0xfb88b1815ea93211ull, 0xfb5d1ee0aa913025ull,
    0xfb3193cc4227c3f4ull, 0xfb061042d6b28e41ull, 0xfada944319b12bcaull, 0xfaaf1fcbbcdd2b40ull};

struct __align__(16) Share {  // what a block tells the others
  uint64_t sum;
  uint32_t count;
  float top;
};
enum Op { kGather, kWeigh, kRefine, kTies, kDone };
struct Message {  // what the first block tells the others
  int op;
  uint32_t lo, hi;   // classes of the first histogram, or keys, of the candidates
  int by_bin;
  int last;          // kGather: the list begins with the order, so the first block draws from it alone
  uint64_t border;   // kTies: how many of the equals are kept; kDone: the last kept token's order
};

struct Shared {
  uint32_t table[1024];  // 2^(-j / 1024) in units of 2^-31
  union {
    struct {
      uint32_t n[kBins], lo[kBins], hi[kBins];  // counts, weights; then their running sums (of later histograms)
    } bins;
    struct {
      uint64_t list[kList], other[kList], sums[kList];
    };
  };
  // running sums of the first histogram over the whole row, up to and including a class
  uint32_t first_n[kBins];
  uint64_t first_w[kBins];
  uint64_t seg_sum[kSegs];
  uint32_t seg_n[kSegs];
  uint64_t warp_w[kWarps];
  uint32_t warp_n[kWarps];
  Share share[2][kMaxCluster];  // of every block, written by it
  Message message[2];
  uint32_t n_list;
  int bin;
  uint32_t found;
};

// ---- order of logits: larger keys are larger logits
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 becomes 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t order_of(uint32_t key, uint32_t index) { return (uint64_t)key << 32 | (0xFFFFFFFFu - index); }
// is it one that can be drawn (no NaN, not -inf)?
__device__ __forceinline__ bool drawable(float x) { return x > -INFINITY; }

// ---- two fp32 operations in one instruction
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- weights
struct Scale {
  float max;     // the largest logit
  float hi, lo;  // log2(e) / temperature
};
__device__ __forceinline__ Scale scale_of(float max, float temperature) {
  Scale s;
  s.max = max;
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;  // log2(e)
  s.hi = kHi / temperature;
  s.lo = (fmaf(-s.hi, temperature, kHi) + kLo) / temperature;
  if (!(s.hi <= FLT_MAX)) {  // (a temperature below 2^-127: differences of logits above 2^-120 count as they should)
    s.hi = FLT_MAX;
    s.lo = 0.f;
  }
  return s;
}
// t is rounded to a multiple of 2^-10 by adding 3 x 2^12: the sum's last bits are that multiple.  The product is in
// the same operation (one rounding), wherever a logit's class is asked for: the compiler is free to join a packed
// product and sum, and steps that did not agree on a class would lose tokens.
constexpr float kRound = 12288.f;
constexpr int kRoundBits = 0x46400000;

// Weights of two logits, and their t in units of 2^-10.  Beyond t = 43, and for -inf and NaN (whose t are as
// large as can be, or NaN, with bits as large), the weight is 0.
__device__ __forceinline__ void weights_of(const Scale& s, const uint32_t* table, float x0, float x1, uint64_t& w0,
                                           uint64_t& w1, int& i0, int& i1) {
  const uint64_t x = pair(x0, x1), m = pair(s.max, s.max), minus = pair(-1.f, -1.f);
  const uint64_t c_hi = pair(s.hi, s.hi), n_hi = pair(-s.hi, -s.hi), n_lo = pair(-s.lo, -s.lo);
  // d + e = max - x exactly
  const uint64_t d = fma2(x, minus, m), b = fma2(m, minus, d);
  const uint64_t e = fma2(add2(x, b), minus, fma2(fma2(b, minus, d), minus, m));
  // t = h - q
  const uint64_t h = mul2(d, c_hi);
  const uint64_t q = fma2(e, n_hi, fma2(d, n_lo, fma2(d, n_hi, h)));
  const uint64_t y = fma2(d, c_hi, pair(kRound, kRound));
  const uint64_t f = fma2(add2(y, pair(-kRound, -kRound)), minus, h);  // exact, at most 2^-11
  const uint64_t r = fma2(q, minus, f);
  // 2^-r = 1 - g, g = u - u^2 / 2 + u^3 / 6, u = r ln 2 < 2^-11.5; the next term is below 2^-50
  constexpr float k1 = 0.693147180559945f, k2 = -0.240226506959101f, k3 = 0.0555041086648216f;
  const uint64_t g = mul2(r, fma2(r, fma2(r, pair(k3, k3), pair(k2, k2)), pair(k1, k1)));
  float y0, y1, g0, g1;
  unpair(y, y0, y1);
  unpair(g, g0, g1);
  i0 = __float_as_int(y0) - kRoundBits;
  i1 = __float_as_int(y1) - kRoundBits;
  const uint32_t a0 = table[__float_as_int(y0) & 1023], a1 = table[__float_as_int(y1) & 1023];
  // a (1 - g) in units of 2^-31: a has its leading bit at 2^30, so that its bits are a float's; the product, at
  // most 2^20, is rounded by adding 3 x 2^22
  const float p0 = fmaf(__uint_as_float(0x4E800000u | (a0 & 0x3FFFFFFFu) >> 7), g0, 12582912.f),
              p1 = fmaf(__uint_as_float(0x4E800000u | (a1 & 0x3FFFFFFFu) >> 7), g1, 12582912.f);
  const uint32_t v0 = a0 + (0x4B400000u - __float_as_uint(p0)), v1 = a1 + (0x4B400000u - __float_as_uint(p1));
  // 2^42 2^-k v 2^-31, rounded
  w0 = ((((uint64_t)v0 << (kBits - 30)) >> min(i0 >> 10, 63)) + 1) >> 1;
  w1 = ((((uint64_t)v1 << (kBits - 30)) >> min(i1 >> 10, 63)) + 1) >> 1;
}
__device__ __forceinline__ uint64_t weight_of(const Scale& s, const uint32_t* table, float x) {
  uint64_t w, unused;
  int i, j;
  weights_of(s, table, x, -INFINITY, w, unused, i, j);
  return w;
}
// t in units of 2^-10, as weights_of has it
__device__ __forceinline__ int log2_below(const Scale& s, float x) {
  return __float_as_int(__fmaf_rn(__fsub_rn(s.max, x), s.hi, kRound)) - kRoundBits;
}
__device__ __forceinline__ void log2_below(const Scale& s, float2 x, int& i0, int& i1) {
  const uint64_t d = fma2(pair(x.x, x.y), pair(-1.f, -1.f), pair(s.max, s.max));
  float y0, y1;
  unpair(fma2(d, pair(s.hi, s.hi), pair(kRound, kRound)), y0, y1);
  i0 = __float_as_int(y0) - kRoundBits;
  i1 = __float_as_int(y1) - kRoundBits;
}
// class of the first histogram; rises as the logit falls
__device__ __forceinline__ int bin_of(int i) { return min(i >> 4, kBins - 1); }
__device__ __forceinline__ int bin_of(const Scale& s, float x) { return bin_of(log2_below(s, x)); }

// x sum, rounded down or up: x is 0 .. 1 or -0, the sum below 2^63 (the product has 24 + 63 bits)
__device__ __forceinline__ uint64_t part_of(float x, uint64_t sum, bool up) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu, e = b >> 23;
  const uint64_t m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
  const int shift = 150 - (int)(e ? e : 1);  // x = m 2^-shift, shift >= 23
  const uint64_t lo = m * sum, hi = __umul64hi(m, sum);
  uint64_t q, rest;
  if (shift < 64) {
    q = hi << (64 - shift) | lo >> shift;
    rest = lo << (64 - shift);
  } else {
    q = shift < 128 ? hi >> (shift - 64) : 0;
    rest = lo | (hi ^ (shift < 128 ? q << (shift - 64) : 0));
  }
  return q + (up && rest ? 1 : 0);
}

// ---- sums
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// of lanes' weights of a few logits each (below 2^44)
__device__ __forceinline__ uint64_t warp_sum_few(uint64_t w) {
  const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)w & 0x3FFFFFu),
                 high = __reduce_add_sync(0xffffffffu, (uint32_t)(w >> 22));
  return ((uint64_t)high << 22) + low;
}
// sums over the block's threads up to and including this one's, of counts and (kWeights) weights
template <bool kWeights>
__device__ void block_scan(uint32_t& n, uint64_t& w, Shared& sh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, n, o);
    const uint64_t b = kWeights ? __shfl_up_sync(0xffffffffu, w, o) : 0ull;
    if (lane >= o) {
      n += a;
      w += b;
    }
  }
  if (lane == 31) {
    sh.warp_n[wid] = n;
    if (kWeights) sh.warp_w[wid] = w;
  }
  __syncthreads();
  n += __reduce_add_sync(0xffffffffu, lane < wid ? sh.warp_n[lane] : 0u);
  if (kWeights) w += warp_sum(lane < wid ? sh.warp_w[lane] : 0ull);
  __syncthreads();
}

// ---- A row's slice in one block of its cluster: pairs of logits, the first of them `skew` in front of the slice
// (so that a pair stands as it does within 16 bytes of the row); logits outside the slice read as -inf.
__device__ __forceinline__ float2 floats(uint2 v, const float*) { return make_float2(__uint_as_float(v.x), __uint_as_float(v.y)); }
__device__ __forceinline__ float2 floats(uint32_t v, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 floats(uint32_t v, const __half*) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
template <class T>
struct Pair {
  using Bits = uint32_t;
};
template <>
struct Pair<float> {
  using Bits = uint2;
};

// kAll: all of the slice is in shared memory.
template <class T, bool kAll>
struct Slice {
  using Bits = typename Pair<T>::Bits;
  const T* x;        // the slice in the row
  int begin, n;      // its first index, its length
  int skew, pairs;   // pairs, with those that begin in front of it or end behind it
  const Bits* room;
  int held;          // so many of the pairs are in shared memory
  bool infinite;     // the row has an infinite logit: such read as 0, all others as -inf
  __device__ __forceinline__ float2 operator()(int i) const {
    if (kAll || i < held) return floats(room[i], x);
    return make_float2(far(2 * i - skew), far(2 * i + 1 - skew));
  }
  __device__ float far(int e) const {
    const float v = e >= 0 && e < n ? (float)x[e] : -INFINITY;
    return !infinite ? v : v == INFINITY ? 0.f : -INFINITY;
  }
  __device__ __forceinline__ int index(int i) const { return begin + 2 * i - skew; }  // of a pair's first logit
};

struct Cluster {
  cg::cluster_group group;
  Shared& sh;
  int rank, size;
  int shares, messages;  // exchanges so far: two buffers each, so that one barrier is enough
  // every block's share; returns the sums over all of them, and over those in front of this one
  __device__ Share exchange(const Share& mine, Share& before) {
    Share* const buf = sh.share[shares++ & 1];
    if ((int)threadIdx.x < size) *group.map_shared_rank(buf + rank, threadIdx.x) = mine;
    group.sync();
    const int lane = threadIdx.x & 31;
    Share s{0, 0, -INFINITY};
    if (lane < size) s = buf[lane];
    Share front{lane < rank ? s.sum : 0, lane < rank ? s.count : 0, 0.f};
#pragma unroll
    for (int o = kMaxCluster / 2; o >= 1; o >>= 1) {
      s.sum += __shfl_xor_sync(0xffffffffu, s.sum, o);
      s.count += __shfl_xor_sync(0xffffffffu, s.count, o);
      s.top = fmaxf(s.top, __shfl_xor_sync(0xffffffffu, s.top, o));
      front.sum += __shfl_xor_sync(0xffffffffu, front.sum, o);
      front.count += __shfl_xor_sync(0xffffffffu, front.count, o);
    }
    before = Share{__shfl_sync(0xffffffffu, front.sum, 0), __shfl_sync(0xffffffffu, front.count, 0), 0.f};
    return Share{__shfl_sync(0xffffffffu, s.sum, 0), __shfl_sync(0xffffffffu, s.count, 0), __shfl_sync(0xffffffffu, s.top, 0)};
  }
  // the first block's message to every block (all threads of it call with the same one); receive() is behind a barrier
  __device__ void send(const Message& m) {
    if ((int)threadIdx.x < size) *group.map_shared_rank(&sh.message[messages & 1], threadIdx.x) = m;
  }
  __device__ Message receive() {
    const Message* const buf = &sh.message[messages++ & 1];
    group.sync();
    return *buf;
  }
};

// Calls f(i, pair) for this thread's pairs of the slice, kAtOnce of them at a time; whole warps together.
template <int kAtOnce, class T, bool kAll, class F>
__device__ __forceinline__ void each_pair(const Slice<T, kAll>& sl, F f) {
  for (int i0 = threadIdx.x & ~31; i0 < sl.pairs; i0 += kThreads * kAtOnce) {
    float2 x[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      const int i = i0 + q * kThreads + (threadIdx.x & 31);
      x[q] = i < sl.pairs ? sl(i) : make_float2(-INFINITY, -INFINITY);
    }
    f(i0 + (threadIdx.x & 31), x);
  }
}

// Adds to a class (lanes without `in` add nothing).
template <bool kWeights>
__device__ __forceinline__ void add_to_bin(Shared& sh, bool in, int b, uint64_t w) {
  if (!in) return;
  atomicAdd(&sh.bins.n[b], 1u);
  if (kWeights) {
    const uint32_t was = atomicAdd(&sh.bins.lo[b], (uint32_t)w), up = (uint32_t)(w >> 32) + (was + (uint32_t)w < was);
    if (up) atomicAdd(&sh.bins.hi[b], up);
  }
}
// The same (all lanes) where a whole warp's elements may be in one class and would queue up.
template <bool kWeights>
__device__ __forceinline__ void add_to_one_bin(Shared& sh, bool in, int b, uint64_t w) {
  const uint32_t lanes = __ballot_sync(0xffffffffu, in);
  if (!lanes) return;
  const int b0 = __shfl_sync(0xffffffffu, b, __ffs(lanes) - 1);
  if (__all_sync(0xffffffffu, !in || b == b0)) {
    const uint64_t sum = kWeights ? warp_sum_few(in ? w : 0ull) : 0ull;
    if ((threadIdx.x & 31) == 0) {
      atomicAdd(&sh.bins.n[b0], __popc(lanes));
      const uint32_t was = atomicAdd(&sh.bins.lo[b0], (uint32_t)sum);
      atomicAdd(&sh.bins.hi[b0], (uint32_t)(sum >> 32) + (was + (uint32_t)sum < was));
    }
  } else {
    add_to_bin<kWeights>(sh, in, b, w);
  }
}
__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins.n[i] = sh.bins.lo[i] = sh.bins.hi[i] = 0;
  __syncthreads();
}

// The first histogram of the slice.  Its last class, most of the logits, is summed up in registers.
template <bool kWeights, class T, bool kAll>
__device__ void first_histogram(const Slice<T, kAll>& sl, const Scale& sc, Shared& sh) {
  constexpr int kAtOnce = 2;
  uint64_t tail_w = 0;
  uint32_t tail_n = 0;
  bool look = true, queue = false;  // a row of logits that lie close (or a high temperature): whole warps in one class
  each_pair<kAtOnce>(sl, [&](int, const float2 (&x)[kAtOnce]) {
    uint64_t w[2 * kAtOnce];
    int b[2 * kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      int i0, i1;
      if (kWeights) {
        weights_of(sc, sh.table, x[q].x, x[q].y, w[2 * q], w[2 * q + 1], i0, i1);
      } else {
        w[2 * q] = w[2 * q + 1] = 0;
        log2_below(sc, x[q], i0, i1);
      }
      b[2 * q] = bin_of(i0);
      b[2 * q + 1] = bin_of(i1);
    }
    if (look) {  // at the warp's first ones
      const int b0 = __shfl_sync(0xffffffffu, b[0], 0);
      queue = __all_sync(0xffffffffu, b[0] == b0);
      look = false;
    }
#pragma unroll
    for (int e = 0; e < 2 * kAtOnce; ++e) {
      const bool tail = b[e] == kBins - 1;
      tail_n += tail && drawable(e & 1 ? x[e / 2].y : x[e / 2].x);
      if (kWeights) tail_w += tail ? w[e] : 0;
    }
    if (queue) {
#pragma unroll
      for (int e = 0; e < 2 * kAtOnce; ++e) add_to_one_bin<kWeights>(sh, b[e] < kBins - 1, b[e], w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 2 * kAtOnce; ++e) add_to_bin<kWeights>(sh, b[e] < kBins - 1, b[e], w[e]);
    }
  });
  tail_n = __reduce_add_sync(0xffffffffu, tail_n);
  if (kWeights) tail_w = warp_sum(tail_w);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&sh.bins.n[kBins - 1], tail_n);
    if (kWeights) {
      const uint32_t was = atomicAdd(&sh.bins.lo[kBins - 1], (uint32_t)tail_w);
      atomicAdd(&sh.bins.hi[kBins - 1], (uint32_t)(tail_w >> 32) + (was + (uint32_t)tail_w < was));
    }
  }
}

// A later one, over the keys lo .. hi, in classes of 2^shift keys from hi down.
template <class T, bool kAll>
__device__ void histogram(const Slice<T, kAll>& sl, const Scale& sc, Shared& sh, uint32_t lo, uint32_t hi, int shift, bool weights) {
  each_pair<1>(sl, [&](int, const float2 (&x)[1]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = e ? x[0].y : x[0].x;
      const uint32_t k = key_of(v);
      const bool in = drawable(v) && k >= lo && k <= hi;
      if (!__any_sync(0xffffffffu, in)) continue;
      const uint64_t w = weights ? weight_of(sc, sh.table, v) : 0;
      add_to_one_bin<true>(sh, in, in ? (int)((hi - k) >> shift) : 0, w);
    }
  });
}

// What the first block knows of the search for a border.
struct Search {
  bool by_weight;     // the goal is a sum of weights (else a count)
  bool weighed;       // the first histogram has weights
  bool first;         // the last histogram is the first one
  uint64_t goal;      // the border is the first token in the order with which the sum reaches it
  uint32_t lo, hi;    // keys of the classes of the last histogram
  int shift;
  uint32_t n_before;  // tokens and weights in front of them
  uint64_t w_before;
};

// The largest key whose class of the first histogram is at least `bin`, or the smallest whose is at most that (a warp
// together): the classes rise as keys fall.
__device__ uint32_t key_at(const Scale& sc, int bin, bool largest) {
  uint32_t lo = kLowestKey, hi = key_of(sc.max);
  const int lane = threadIdx.x & 31;
  if (!largest && bin_of(sc, value_of(lo)) <= bin) return lo;
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 32 + 1;  // probes lo + step, lo + 2 step, ...
    const uint64_t at = (uint64_t)lo + (uint64_t)step * (lane + 1);
    const bool in = at <= hi;
    const int b = in ? bin_of(sc, value_of((uint32_t)at)) : 0;
    if (largest) {  // true for the keys up to the one sought
      const int n = __popc(__ballot_sync(0xffffffffu, in && b >= bin));
      hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)step * (n + 1) - 1);
      lo += step * n;
    } else {  // lo's class is above, hi's is not
      const int n = __popc(__ballot_sync(0xffffffffu, in && b > bin));
      hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)step * (n + 1));
      lo += step * n;
      if (hi - lo <= 1) return hi;
    }
  }
  return lo;
}

// The first block: sums the cluster's histograms, some neighbouring classes a thread, as running sums.
__device__ void merge(Cluster& cl, Shared& sh, bool first, bool weights) {
  constexpr int kPairs = kBinsPerThread / 2;
  uint32_t n[kBinsPerThread];
  uint64_t w[kBinsPerThread];
#pragma unroll
  for (int q = 0; q < kBinsPerThread; ++q) n[q] = 0, w[q] = 0;
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which > 0 && !weights) break;
#pragma unroll
    for (int h = 0; h < kPairs; ++h) {
      uint2 v[kMaxCluster];  // all blocks' loads travel together
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        v[r] = make_uint2(0u, 0u);
        if (r < cl.size) {
          const Shared* const o = cl.group.map_shared_rank(&sh, r);
          v[r] = reinterpret_cast<const uint2*>(which == 0 ? o->bins.n : which == 1 ? o->bins.lo : o->bins.hi)[threadIdx.x * kPairs + h];
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (which == 0) {
          n[2 * h] += v[r].x;
          n[2 * h + 1] += v[r].y;
        } else {
          w[2 * h] += (uint64_t)v[r].x << (which == 2 ? 32 : 0);
          w[2 * h + 1] += (uint64_t)v[r].y << (which == 2 ? 32 : 0);
        }
      }
    }
  }
  uint32_t tn = 0;
  uint64_t tw = 0;
#pragma unroll
  for (int q = 0; q < kBinsPerThread; ++q) {
    tn += n[q];
    tw += w[q];
  }
  if (weights) block_scan<true>(tn, tw, sh);
  else block_scan<false>(tn, tw, sh);  // (its barriers: everybody has read this block's own counts)
#pragma unroll
  for (int q = kBinsPerThread - 1; q >= 0; --q) {
    const int b = threadIdx.x * kBinsPerThread + q;
    if (first) {
      sh.first_n[b] = tn;
      sh.first_w[b] = tw;
    } else {
      sh.bins.n[b] = tn;
      sh.bins.lo[b] = (uint32_t)tw;
      sh.bins.hi[b] = (uint32_t)(tw >> 32);
    }
    tn -= n[q];
    tw -= w[q];
  }
  __syncthreads();
}

// The first place of rising running sums cum(0) .. cum(n - 1) that reaches the goal (the block together).
template <class F>
__device__ int reaches(int n, uint64_t goal, Shared& sh, F cum) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (cum(i) >= goal && (i == 0 || cum(i - 1) < goal)) sh.bin = i;
  __syncthreads();
  const int b = sh.bin;
  __syncthreads();
  return b;
}

// The first block: what to do about the class that holds the border.
__device__ Message next_step(Search& s, const Scale& sc, Shared& sh) {
  auto cum_n = [&](int i) { return s.first ? sh.first_n[i] : sh.bins.n[i]; };
  auto cum_w = [&](int i) { return s.first ? sh.first_w[i] : (uint64_t)sh.bins.hi[i] << 32 | sh.bins.lo[i]; };
  const int b = s.by_weight ? reaches(kBins, s.goal - s.w_before, sh, cum_w) : reaches(kBins, s.goal - s.n_before, sh, cum_n);
  const uint32_t upto = cum_n(b), in_front = b ? cum_n(b - 1) : 0u;
  const uint64_t w_front = b ? cum_w(b - 1) : 0;
  Message m{};
  if (s.first && upto <= kList) {  // with all in front: a limit to the rest of top-k is among them, too
    m.op = kGather;
    m.by_bin = 1;
    m.hi = (uint32_t)b;
  } else if (!s.weighed) {
    m.op = kWeigh;  // a long list of top-k's: what top-p keeps of it takes the first histogram's weights
  } else {
    const bool first = s.first;
    s.n_before += in_front;
    s.w_before += w_front;
    if (first && upto - in_front <= kList) {
      m.op = kGather;
      m.by_bin = 1;
      m.lo = m.hi = (uint32_t)b;
    } else {
      if (first) {
        m.hi = key_at(sc, b, true);
        m.lo = key_at(sc, b, false);
      } else {
        m.hi = s.hi - ((uint32_t)b << s.shift);
        m.lo = max(s.lo, m.hi - ((1u << s.shift) - 1u));
      }
      if (upto - in_front <= kList) {
        m.op = kGather;
      } else if (m.lo == m.hi) {
        m.op = kTies;
        const uint64_t w = weight_of(sc, sh.table, value_of(m.lo));
        m.border = s.by_weight ? (s.goal - s.w_before + w - 1) / w : s.goal - s.n_before;
      } else {
        m.op = kRefine;
        s.first = false;
        s.lo = m.lo;
        s.hi = m.hi;
        s.shift = max(0, 22 - __clz(m.hi - m.lo));
      }
    }
  }
  m.last = m.op == kGather && s.n_before == 0;
  __syncthreads();  // (the running sums may give way to a list)
  return m;
}

// The first block: its list of n candidates in falling order, with the running sums of their weights.
__device__ void sort_list(const Scale& sc, Shared& sh, int n) {
  static_assert(kList <= kThreads, "");
  const int i = threadIdx.x;
  uint64_t mine = 0;
  if (i < n) {
    mine = sh.list[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += sh.list[j] > mine;
    sh.other[place] = mine;
  }
  __syncthreads();
  uint64_t w = 0;
  uint32_t unused = 0;
  if (i < n) {
    mine = sh.other[i];
    w = weight_of(sc, sh.table, value_of((uint32_t)(mine >> 32)));
    sh.list[i] = mine;
  }
  block_scan<true>(unused, w, sh);
  if (i < n) sh.sums[i] = w;
  __syncthreads();
}

// Sums of a slice by segment in the order of the index.  Of the logits from `last` up (of those that equal it the ones up
// to an index) weigh(x, w) gives two logits' weights and how many of them count after all.  Few of a row's logits do,
// as a rule: each lane first marks those of its pairs, then weighs them two at a time.  Afterwards `find` gives the
// index with which the sum over the row exceeds `target`.
struct Border {
  float last;
  int last_index;
  __device__ __forceinline__ bool in(float x, int index) const { return x > last || (x == last && index <= last_index); }
};
constexpr int kStep = 16;  // pairs of a lane at a time, a bit for each logit
template <class T, bool kAll>
__device__ __forceinline__ int segment_pairs(const Slice<T, kAll>& sl) {
  return ((sl.pairs + kSegs - 1) / kSegs + 32 * kStep - 1) / (32 * kStep) * (32 * kStep);
}
template <class T, bool kAll, class Weigh>
__device__ Share segments(const Slice<T, kAll>& sl, Shared& sh, Cluster& cl, Share& before, const Border& border,
                          Weigh weigh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int len = segment_pairs(sl);
  for (int s = wid; s < kSegs; s += kWarps) {
    uint64_t w = 0;
    uint32_t n = 0;
    const int end = min(sl.pairs, (s + 1) * len);
    for (int i0 = s * len; i0 < end; i0 += 32 * kStep) {
      uint32_t marks = 0;
      // (the equals are all in or all out but in one step of a row)
      const int i_first = sl.index(i0), i_last = sl.index(i0 + 32 * kStep);
      if (i_last <= border.last_index || i_first > border.last_index) {
        const bool equals = i_last <= border.last_index;
#pragma unroll
        for (int q = 0; q < kStep; ++q) {
          const int i = i0 + 32 * q + lane;
          const float2 x = i < end ? sl(i) : make_float2(-INFINITY, -INFINITY);
          const bool a = x.x > border.last || (equals && x.x == border.last), c = x.y > border.last || (equals && x.y == border.last);
          marks |= (a ? 1u << (2 * q) : 0u) | (c ? 2u << (2 * q) : 0u);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < kStep; ++q) {
          const int i = i0 + 32 * q + lane;
          const float2 x = i < end ? sl(i) : make_float2(-INFINITY, -INFINITY);
          marks |= ((uint32_t)border.in(x.x, sl.index(i)) | (uint32_t)border.in(x.y, sl.index(i) + 1) << 1) << (2 * q);
        }
      }
      while (__any_sync(0xffffffffu, marks != 0)) {
        float2 x = make_float2(-INFINITY, -INFINITY);
        if (marks) {
          const int e = __ffs(marks) - 1;
          marks &= marks - 1;
          const float2 v = sl(i0 + 32 * (e >> 1) + lane);
          x.x = e & 1 ? v.y : v.x;
        }
        if (marks) {
          const int e = __ffs(marks) - 1;
          marks &= marks - 1;
          const float2 v = sl(i0 + 32 * (e >> 1) + lane);
          x.y = e & 1 ? v.y : v.x;
        }
        uint64_t a, b;
        n += weigh(x, a, b);
        w += a + b;
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    w = __any_sync(0xffffffffu, w != 0) ? warp_sum(w) : 0;
    if (lane == 0) {
      sh.seg_sum[s] = w;
      sh.seg_n[s] = n;
    }
  }
  __syncthreads();
  if (wid == 0) {  // running sums over the segments, four to a lane
    static_assert(kSegs == 128, "");
    uint64_t v[4], sum = 0;
    uint32_t n = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = sum += sh.seg_sum[4 * lane + q];
      n += sh.seg_n[4 * lane + q];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    uint64_t up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sh.seg_sum[4 * lane + q] = v[q] + up - sum;
    if (lane == 31) {
      sh.warp_w[0] = up;
      sh.warp_n[0] = n;
    }
  }
  __syncthreads();
  return cl.exchange(Share{sh.warp_w[0], sh.warp_n[0], 0.f}, before);
}
// (in the slice, for all threads of the block that holds it; else -1)
template <class T, bool kAll, class Weigh>
__device__ int find(const Slice<T, kAll>& sl, Shared& sh, const Share& before, uint64_t target, const Border& border,
                    Weigh weigh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (target < before.sum || target - before.sum >= sh.seg_sum[kSegs - 1]) return -1;
  const uint64_t rest = target - before.sum;
  int s = 0;
#pragma unroll
  for (int c = 0; c < kSegs; c += 32) s += __popc(__ballot_sync(0xffffffffu, sh.seg_sum[c + lane] <= rest));
  const int len = segment_pairs(sl);
  uint64_t sum = s ? sh.seg_sum[s - 1] : 0;
  const int end = min(sl.pairs, (s + 1) * len);
  for (int c = s * len; c < end; c += kThreads) {  // a pair of the segment to a thread
    const int i = c + (int)threadIdx.x;
    float2 x = i < end ? sl(i) : make_float2(-INFINITY, -INFINITY);
    if (!border.in(x.x, sl.index(i))) x.x = -INFINITY;
    if (!border.in(x.y, sl.index(i) + 1)) x.y = -INFINITY;
    uint64_t a, b;
    weigh(x, a, b);
    const uint64_t mine = warp_sum_few(a + b);
    if (lane == 0) sh.warp_w[wid] = mine;
    __syncthreads();
    const uint64_t w = lane < kWarps ? sh.warp_w[lane] : 0, front = sum + warp_sum(lane < wid ? w : 0), all = warp_sum(w);
    if (front <= rest && rest < front + mine) {
      uint64_t upto = a + b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      // the first lane that exceeds, and of its pair the second logit if the sum without it does not
      const uint32_t over = __ballot_sync(0xffffffffu, front + upto > rest);
      if (lane == __ffs(over) - 1) sh.found = (uint32_t)(2 * i - sl.skew + (front + upto - b <= rest));
    }
    __syncthreads();
    if (rest < sum + all) return (int)sh.found;
    sum += all;
  }
  return -1;
}

// The index of the m-th logit (from 1) that equals v.
template <class T, bool kAll>
__device__ uint32_t tie(const Slice<T, kAll>& sl, Shared& sh, Cluster& cl, float v, uint64_t m) {
  const Border up{v, INT_MAX};  // (larger ones are marked, too, and weigh nothing)
  auto one = [&](float2 x, uint64_t& a, uint64_t& b) {
    a = x.x == v;
    b = x.y == v;
    return (uint32_t)(a + b);
  };
  Share before, unused;
  segments(sl, sh, cl, before, up, one);
  const int i = find(sl, sh, before, m - 1, up, one);
  return cl.exchange(Share{0, i >= 0 ? (uint32_t)(sl.begin + i) + 1u : 0u, 0.f}, unused).count - 1u;
}

// the larger of each half's elements; NaN counts for nothing
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, const float*) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, const __nv_bfloat16*) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, const __half*) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <class T>
__device__ __forceinline__ float largest_of(uint32_t a, const T* t) {
  const float2 f = floats(a, t);
  return fmaxf(f.x, f.y);
}
__device__ __forceinline__ float largest_of(uint32_t a, const float*) { return __uint_as_float(a); }
// -inf in every element
template <class T>
constexpr uint32_t kNothing = sizeof(T) == 4 ? 0xFF800000u : 0u;
template <>
constexpr uint32_t kNothing<__nv_bfloat16> = 0xFF80FF80u;
template <>
constexpr uint32_t kNothing<__half> = 0xFC00FC00u;

// What the calls of a row have in common.
struct Row {
  float temperature, top_p, min_p, random;
  int top_k;
  __device__ bool fine() const {
    return temperature >= 0.f && temperature < INFINITY && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f &&
           min_p <= 1.f && random >= 0.f && random <= 1.f;
  }
};

template <class T, bool kAll>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) sample_kernel(const SampleArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint4* const room = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  Cluster cl{cg::this_cluster(), sh, 0, 0, 0, 0};
  cl.rank = (int)cl.group.block_rank();
  cl.size = (int)cl.group.num_blocks();
  // (no block writes to another's shared memory before that one has begun: the wait is in front of the first exchange)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row = (int)(blockIdx.x / (unsigned)cl.size);
  Row r;
  r.temperature = p.temperature ? p.temperature[row] : 1.f;
  r.top_k = p.top_k ? p.top_k[row] : 0;
  r.top_p = p.top_p ? p.top_p[row] : 1.f;
  r.min_p = p.min_p ? p.min_p[row] : 0.f;
  r.random = p.random[row];

  // ---- the slice to shared memory, and its largest logit
  Slice<T, kAll> sl;
  sl.begin = min(p.vocab, cl.rank * p.slice);
  sl.n = min(p.vocab, sl.begin + p.slice) - sl.begin;
  sl.x = static_cast<const T*>(p.logits) + row * p.stride + sl.begin;
  constexpr int kVec = 16 / sizeof(T);
  sl.skew = (int)((reinterpret_cast<uintptr_t>(sl.x) & 15) / sizeof(T));
  sl.room = reinterpret_cast<const typename Slice<T, kAll>::Bits*>(room);
  const int vecs = (sl.skew + sl.n + kVec - 1) / kVec;
  sl.pairs = (sl.skew + sl.n + 1) / 2;
  sl.held = min(sl.pairs, p.room * (kVec / 2));
  sl.infinite = false;
  uint32_t most = kNothing<T>;
  {
    const uint4* const base = reinterpret_cast<const uint4*>(sl.x - sl.skew);
    constexpr int kAtOnce = 8;
    const uint64_t fine = __ldg(c_fine + lane);
    for (int v0 = tid; v0 < vecs || v0 == tid; v0 += kThreads * kAtOnce) {
      uint4 v[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int j = v0 + q * kThreads, e = j * kVec - sl.skew;  // first element
        v[q] = make_uint4(kNothing<T>, kNothing<T>, kNothing<T>, kNothing<T>);
        if (e >= 0 && e + kVec <= sl.n) {
          v[q] = __ldg(base + j);
        } else if (j < vecs) {  // the slice's ends
          for (int i = 0; i < kVec; ++i)
            if (e + i >= 0 && e + i < sl.n) {
              uint32_t& to = (&v[q].x)[i * sizeof(T) / 4];
              if constexpr (sizeof(T) == 4) to = __float_as_uint(sl.x[e + i]);
              else to = __byte_perm(to, reinterpret_cast<const uint16_t*>(sl.x)[e + i], i & 1 ? 0x5410 : 0x3254);
            }
        }
      }
      if (v0 == tid) {  // while the first ones travel
        for (int i = tid; i < 1024; i += kThreads)
          sh.table[i] = (uint32_t)min((__umul64hi(c_coarse[i >> 5], fine) + 0x80000000ull) >> 32, 0x7FFFFFFFull);
        clear_bins(sh);
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int j = v0 + q * kThreads;
        if (j < vecs && j < p.room) room[j] = v[q];
        most = larger(larger(larger(most, v[q].x, sl.x), v[q].y, sl.x), larger(v[q].z, v[q].w, sl.x), sl.x);
      }
    }
  }
  float top = largest_of(most, sl.x);
  uint32_t top_key = drawable(top) ? key_of(top) : 0u;
  top_key = __reduce_max_sync(0xffffffffu, top_key);
  if (lane == 0) sh.warp_n[wid] = top_key;
  __syncthreads();
  top_key = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.warp_n[lane] : 0u);
  top = top_key ? value_of(top_key) : -INFINITY;
  Share before;
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  top = cl.exchange(Share{0, 0, top}, before).top;
  if (!drawable(top) || !r.fine()) {
    if (cl.rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.probs) p.probs[row] = 0.f;
      if (p.kept) p.kept[row] = 0;
    }
    cl.group.sync();  // a block's shared memory stays until the others have read it
    return;
  }

  if (top == INFINITY) {  // the infinite ones share it all
    T* const x = reinterpret_cast<T*>(room);
    for (int i = tid; i < 2 * sl.held; i += kThreads) x[i] = (T)((float)x[i] == INFINITY ? 0.f : -INFINITY);
    sl.infinite = true;
    top = 0.f;
    __syncthreads();
  }

  // ---- the order's border: the last token that top-k and top-p keep
  const bool greedy = r.temperature == 0.f;
  const Scale sc = scale_of(top, greedy ? 1.f : r.temperature);
  const uint64_t least = part_of(r.min_p, kOne, true);  // min-p's weight
  auto target_of = [&](uint64_t sum) { return min(sum - 1, part_of(r.random, sum, false)); };
  auto write = [&](int token, uint32_t n, float x, uint64_t sum) {
    p.tokens[row] = token;
    if (p.kept) p.kept[row] = (int32_t)n;
    if (p.probs) {
      // (the weight as a number: its multiple of 2^-42 may have few bits)
      const float d = sc.max - x, b = d - sc.max, e = (sc.max - (d - b)) - (x + b);
      const float h = d * sc.hi, l = fmaf(d, sc.hi, -h) + fmaf(d, sc.lo, e * sc.hi);
      p.probs[row] = exp2f(-h) * (1.f - 0.6931471805599453f * l) * ((float)kOne / (float)sum);
    }
  };
  uint64_t border = 0;
  if (greedy) {
    const uint32_t index = tie(sl, sh, cl, top, 1);
    if (cl.rank == 0 && tid == 0) write((int)index, 1u, top, kOne);
    cl.group.sync();  // a block's shared memory stays until the others have read it
    return;
  }
  {
    const bool by_count = r.top_k > 0 && r.top_k < p.vocab, by_weight = r.top_p < 1.f;
    if (by_count || by_weight) {
      // (weights with the counts only where there is no top-k: its candidates are few, as a rule, and are weighed
      // in their list)
      if (by_count) first_histogram<false>(sl, sc, sh);
      else first_histogram<true>(sl, sc, sh);
      cl.group.sync();
      Search se{};  // (of use in the first block)
      auto restart = [&](uint64_t whole) {  // top-p of what top-k keeps, from the first histogram on
        se.by_weight = se.first = true;
        se.goal = max((uint64_t)1, part_of(r.top_p, whole, true));
        se.n_before = 0;
        se.w_before = 0;
      };
      if (cl.rank == 0) {
        merge(cl, sh, true, !by_count);
        se.weighed = !by_count || !by_weight;
        if (tid == 0) sh.n_list = 0;
        if (by_count && (uint32_t)r.top_k < sh.first_n[kBins - 1]) {
          se.first = true;
          se.goal = (uint64_t)r.top_k;
        } else if (by_weight && !by_count) {
          restart(sh.first_w[kBins - 1]);
        }
        if (se.first) cl.send(next_step(se, sc, sh));
        else cl.send(Message{by_weight ? kWeigh : kDone, 0, 0, 0, 0, 0});  // top-k keeps all
      }
      for (;;) {
        const Message m = cl.receive();
        if (m.op == kDone) {
          border = m.border;
          break;
        }
        if (m.op == kGather) {
          Shared* const to = cl.group.map_shared_rank(&sh, 0);
          constexpr int kAtOnce = 4;
          // (a class is a range of t in units of 2^-10, the last one without an end)
          const uint32_t lo = m.by_bin ? m.lo * 16u : m.lo;
          const uint32_t range = (m.by_bin ? m.hi == kBins - 1 ? 0x7FFFFFFFu : m.hi * 16u + 15u : m.hi) - lo;
          each_pair<kAtOnce>(sl, [&](int i, const float2 (&x)[kAtOnce]) {
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
              int c[2];
              log2_below(sc, x[q], c[0], c[1]);
              if (!m.by_bin) {
                c[0] = (int)key_of(x[q].x);
                c[1] = (int)key_of(x[q].y);
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v = e ? x[q].y : x[q].x;
                if ((uint32_t)c[e] - lo <= range && drawable(v)) {
                  const uint32_t at = atomicAdd(&to->n_list, 1u);
                  if (at < kList) to->list[at] = order_of(key_of(v), (uint32_t)(sl.index(i + q * kThreads) + e));
                }
              }
            }
          });
          cl.group.sync();
          if (m.last && cl.rank != 0) return;  // (the first block reads nothing of the others' any more)
          if (cl.rank == 0) {
            const int n = (int)min(sh.n_list, (uint32_t)kList);
            sort_list(sc, sh, n);
            auto sums = [&](int i) { return sh.sums[i]; };
            int at = se.by_weight ? reaches(n, se.goal - se.w_before, sh, sums) : (int)(se.goal - se.n_before) - 1;
            bool done = true;
            if (!se.by_weight && by_weight) {
              const uint64_t w_front = se.w_before;
              restart(w_front + sh.sums[at]);
              done = se.goal > w_front;  // (else in front of these)
              if (done) at = reaches(n, se.goal - w_front, sh, sums);
            }
            if (m.last) {
              // the list begins with the order: the draw is among its first ones
              const uint64_t mine = tid <= at ? sh.list[tid] : 0;
              uint64_t w = tid <= at ? sh.sums[tid] - (tid ? sh.sums[tid - 1] : 0) : 0;
              const int n_kept = __syncthreads_count(tid <= at && w >= least);
              const uint64_t sum = sh.sums[n_kept - 1], target = target_of(sum);
              if (tid < n_kept) {  // by index (the order's lower half falls with it)
                int place = 0;
                for (int j = 0; j < n_kept; ++j) place += (uint32_t)sh.list[j] > (uint32_t)mine;
                sh.other[place] = (uint64_t)tid << 48 | w;
              }
              __syncthreads();
              w = tid < n_kept ? sh.other[tid] : 0;
              const int from = (int)(w >> 48);
              uint64_t upto = w &= 0xFFFFFFFFFFFFull;
              uint32_t unused = 0;
              block_scan<true>(unused, upto, sh);
              if (tid < n_kept && upto > target && upto - w <= target) {
                const uint64_t it = sh.list[from];
                write((int)(0xFFFFFFFFu - (uint32_t)it), (uint32_t)n_kept, value_of((uint32_t)(it >> 32)), sum);
              }
              return;
            }
            if (done) {
              cl.send(Message{kDone, 0, 0, 0, 0, sh.list[at]});
            } else {
              if (tid == 0) sh.n_list = 0;
              cl.send(next_step(se, sc, sh));
            }
          }
        } else if (m.op == kWeigh) {
          clear_bins(sh);
          first_histogram<true>(sl, sc, sh);
          cl.group.sync();
          if (cl.rank == 0) {
            merge(cl, sh, true, true);
            se.weighed = true;
            if (!se.first) restart(sh.first_w[kBins - 1]);
            cl.send(next_step(se, sc, sh));
          }
        } else if (m.op == kRefine) {
          clear_bins(sh);
          histogram(sl, sc, sh, m.lo, m.hi, max(0, 22 - __clz(m.hi - m.lo)), by_weight);
          cl.group.sync();
          if (cl.rank == 0) {
            merge(cl, sh, false, by_weight);
            cl.send(next_step(se, sc, sh));
          }
        } else {
          const float v = value_of(m.lo);
          const uint32_t index = tie(sl, sh, cl, v, m.border);
          if (cl.rank == 0) {
            bool done = true;
            if (!se.by_weight && by_weight) {
              const uint64_t w = weight_of(sc, sh.table, v), w_front = se.w_before;
              restart(w_front + m.border * w);
              done = se.goal > w_front;
              if (done) cl.send(Message{kTies, m.lo, m.lo, 0, 0, (se.goal - w_front + w - 1) / w});
            } else {
              cl.send(Message{kDone, 0, 0, 0, 0, order_of(m.lo, index)});
            }
            if (!done) cl.send(next_step(se, sc, sh));
          }
        }
      }
    }
  }

  // ---- the draw among the tokens up to the border, and with min-p's weight
  const Border kept{border ? value_of((uint32_t)(border >> 32)) : -INFINITY,  // the border's logit and index
                    border ? (int)(0xFFFFFFFFu - (uint32_t)border) : INT_MIN};
  auto weigh = [&](float2 x, uint64_t& a, uint64_t& b) {
    int i0, i1;
    weights_of(sc, sh.table, x.x, x.y, a, b, i0, i1);
    const bool in0 = drawable(x.x) && a >= least, in1 = drawable(x.y) && b >= least;
    a = in0 ? a : 0;
    b = in1 ? b : 0;
    return (uint32_t)in0 + (uint32_t)in1;
  };
  const Share sum = segments(sl, sh, cl, before, kept, weigh);
  const int i = find(sl, sh, before, target_of(sum.sum), kept, weigh);
  if (i >= 0 && tid == 0) {
    const float2 x = sl((i + sl.skew) >> 1);
    write(sl.begin + i, sum.count, (i + sl.skew) & 1 ? x.y : x.x, sum.sum);
  }
  cl.group.sync();  // a block's shared memory stays until the others have read it
}

template <class T, bool kAll>
cudaError_t launch_as(const SampleArgs& p, int blocks, size_t smem, int most_smem, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit for this kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(sample_kernel<T, kAll>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)p.n_rows * blocks);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, sample_kernel<T, kAll>, p);
}

template <class T>
cudaError_t launch(SampleArgs p, int sms, int most_smem, cudaStream_t s) {
  // Blocks per row: more of them while the rows alone leave SMs idle or a slice is so large that only one
  // block fits an SM; a slice has at least 2,048 logits (a cluster's barriers cost what its blocks save).
  // With 2, 4 and 8 blocks: one row of 32,003 logits 16.7, 14.6 and 12.6 us, 64 rows of 131,072 170, 79 and 61,
  // 500 rows of 50,021 in 16 bits 159, 210 and 336; the rule takes 8, 8 and 2.
  const int fixed = (int)(sizeof(Shared) + 15) / 16 * 16;
  constexpr int kLeast = 2048, kShare = 224 * 1024 / kBlocksPerSm;
  int blocks = 1;
  while (blocks < kMaxCluster && p.vocab / blocks >= 2 * kLeast &&
         ((int64_t)p.n_rows * blocks < sms || fixed + ((p.vocab - 1) / blocks + 1) * (int)sizeof(T) > kShare))
    blocks *= 2;
  p.slice = (p.vocab - 1) / blocks + 1;
  constexpr int kVec = 16 / sizeof(T);
  const int need = (p.slice + 2 * kVec - 2) / kVec;
  p.room = std::min(need, (most_smem - fixed) / 16);
  const size_t smem = fixed + 16 * (size_t)p.room;
  return p.room == need ? launch_as<T, true>(p, blocks, smem, most_smem, s)
                        : launch_as<T, false>(p, blocks, smem, most_smem, s);
}
}  // namespace

cudaError_t launch_sample(const SampleArgs& p, int dtype, int sms, cudaStream_t s) {
  constexpr int kSmem = 227 * 1024;
  if (dtype == MSM_FP32) return launch<float>(p, sms, kSmem, s);
  return dtype == MSM_BF16 ? launch<__nv_bfloat16>(p, sms, kSmem, s) : launch<__half>(p, sms, kSmem, s);
}

}  // namespace msm
