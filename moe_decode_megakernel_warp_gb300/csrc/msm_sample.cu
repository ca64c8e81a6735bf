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
// definition in 64-bit floating point but for the weights' own rounding.  That matters: a row's 100,000
// borders between tokens lie so close that sums in 32-bit floating point draw another token once in some
// thousand rows.  exp2 is computed to 2^-42: the argument as two floats, its leading 10 fractional bits
// through a table of 1,024 entries (products of two 64-bit constants), the rest by a polynomial
// of third degree.
//
// A row belongs to one cluster of up to eight blocks, each with a slice of it in shared memory, so the
// logits are read once.  The order's border is found without sorting the row: a histogram over 1,024
// classes of the scaled logit (counts and, where top-p needs them, weights), of which only the class that
// holds the border goes on: gathered and sorted by the cluster's first block when it is small (top-k: with all
// classes in front of it), else divided into 1,024 finer classes, down to single values, whose equals are
// told apart by index.  Between the steps the blocks exchange sums through distributed shared memory.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "msm_attn.cuh"
#include "msm_sample.h"

namespace cg = cooperative_groups;

namespace msm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr float kBinsPerLog2 = 16.f;  // classes of the first histogram per factor of two of the weight
constexpr int kList = 1024;           // candidates that are sorted
constexpr int kSegs = 128;            // segments of a slice, in the order of the index
constexpr int kMaxCluster = 8;
constexpr int kOneBits = 42;          // a weight of 1
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
__constant__ uint64_t c_fine[32] = {
    0xffffffffffffffffull, 0xffd3a751c0f7e10cull, 0xffa756521c8daed2ull, 0xff7b0cffbe159675ull,
    0xff4ecb59511ec8a5ull, 0xff22915d81736f63ull, 0xfef65f0afb18a3caull, 0xfeca34606a4e63dcull,
    0xfe9e115c7b8f884cull, 0xfe71f5fddb91ba4bull, 0xfe45e2433745695dull, 0xfe19d62b3bd5c123ull,
    0xfdedd1b496a89f35ull, 0xfdc1d4ddf55e88f3ull, 0xfd95dfa605d2a15eull, 0xfd69f20b761a9ef0ull,
    0xfd3e0c0cf486c175ull, 0xfd122da92fa1c7e8ull, 0xfce656ded630e654ull, 0xfcba87ac9733bbafull,
    0xfc8ec01121e447bbull, 0xfc63000b25b6e0f0ull, 0xfc374799525a2a57ull, 0xfc0b96ba57b7097bull,
    0xfbdfed6ce5f09c49ull, 0xfbb44bafad642efdull, 0xfb88b1815ea93211ull, 0xfb5d1ee0aa913025ull,
    0xfb3193cc4227c3f4ull, 0xfb061042d6b28e41ull, 0xfada944319b12bcaull, 0xfaaf1fcbbcdd2b40ull};

struct Share {  // what a block tells the others
  uint64_t sum;
  uint32_t count, top;
};
enum Op { kGather, kRefine, kTies, kDone };
struct Message {  // what the first block tells the others
  int op;
  uint32_t lo, hi;   // keys of the candidates
  uint64_t border;   // kTies: how many of the equals are kept; kDone: the last kept token's order
};

struct Shared {
  uint64_t table[1024];
  union {
    struct {
      uint32_t n[kBins], lo[kBins], hi[kBins];
    } bins;
    uint64_t list[kList];
  };
  // sums up to and including a class, of the whole row: of the first histogram, of the last one or of the list
  uint32_t first_n[kBins], last_n[kBins];
  uint64_t first_w[kBins], last_w[kBins];
  uint64_t seg_sum[kSegs];
  uint32_t seg_n[kSegs];
  uint64_t warp_w[kWarps];
  uint32_t warp_n[kWarps], warp_top[kWarps];
  Share share[2];
  Message message[2];
  uint32_t n_list;
  int bin;
  uint32_t found;
};

// ---- order of logits: larger keys are larger logits; 0: never drawn (-inf, NaN)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 becomes 0)
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t order_of(uint32_t key, uint32_t index) { return (uint64_t)key << 32 | (0xFFFFFFFFu - index); }

// ---- weights
struct Scale {
  uint32_t top;  // key of the largest logit
  float max;     // and its value
  float hi, lo;  // log2(e) / temperature
};
__device__ __forceinline__ Scale scale_of(uint32_t top, float temperature) {
  Scale s;
  s.top = top;
  s.max = value_of(top);
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;  // log2(e)
  s.hi = kHi / temperature;
  s.lo = (fmaf(-s.hi, temperature, kHi) + kLo) / temperature;
  return s;
}
// (max - x) log2(e) / T as hi + lo; hi is infinite (and lo means nothing) where the difference is
__device__ __forceinline__ void log2_below(const Scale& s, uint32_t key, float& hi, float& lo) {
  const float x = value_of(key);
  const float d = s.max - x, b = d - s.max, e = (s.max - (d - b)) + (-x - b);  // d + e = max - x exactly
  hi = d * s.hi;
  lo = fmaf(d, s.hi, -hi) + fmaf(d, s.lo, e * s.hi);
}
// 2^42 exp((x - max) / T), rounded
__device__ __forceinline__ uint64_t weight_of(const Scale& s, const uint64_t* table, uint32_t key) {
  if (key == s.top) return 1ull << kOneBits;
  float h, l;
  log2_below(s, key, h, l);
  if (!(h < 43.f)) return 0;
  const int n = __float2int_rz(h * 1024.f);
  const float f = fmaf((float)n, -1.f / 1024.f, h);  // exact: 0 <= f < 2^-10
  const float r = f + l, rl = (f - r) + l;
  // 2^-r = 1 - (u - u^2 / 2 + u^3 / 6 - ...), u = r ln 2 < 2^-10.5; the next term is below 2^-46
  constexpr float kHi = 0.693147182464599609375f, kLo = -1.904654299957768e-9f;  // ln 2
  const float u = r * kHi, ul = fmaf(r, kHi, -u) + fmaf(r, kLo, rl * kHi);
  const float g = ul - u * u * fmaf(u, -1.f / 6.f, 0.5f);
  const int qu = __float2int_rn(u * 0x1p41f);
  const int64_t q = 2 * (int64_t)qu + __float2int_rn((g + fmaf((float)qu, -0x1p-41f, u)) * 0x1p42f);
  const uint64_t a = table[n & 1023];
  const int64_t less = (int64_t)((a + 0x80000000ull) >> 32) * q;  // 2^-31 x 2^-42
  const int shift = 63 - kOneBits + (n >> 10);
  return (a - (uint64_t)(less >> 10) + (1ull << (shift - 1))) >> shift;
}

// class of the first histogram; rises as the key falls
__device__ __forceinline__ int bin_of(const Scale& s, uint32_t key) {
  if (key == s.top) return 0;
  const float z = (s.max - value_of(key)) * (s.hi * kBinsPerLog2);
  return (int)min(__float2uint_rz(z), (uint32_t)kBins - 1u);
}

// ---- a block's sums
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// sums over the block's threads up to and including this one's
__device__ void block_scan(uint32_t& n, uint64_t& w, Shared& sh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, n, o);
    const uint64_t b = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) {
      n += a;
      w += b;
    }
  }
  if (lane == 31) {
    sh.warp_n[wid] = n;
    sh.warp_w[wid] = w;
  }
  __syncthreads();
  for (int i = 0; i < wid; ++i) {
    n += sh.warp_n[i];
    w += sh.warp_w[i];
  }
  __syncthreads();
}

// A row's slice in one block of its cluster, and the steps that all blocks take together.
template <class T>
struct Slice {
  const T* x;        // the row
  int begin, n;      // the slice's first index, its length
  const uint32_t* keys;
  int held;          // so many of its keys are in shared memory
  __device__ __forceinline__ uint32_t key(int i) const {
    return i < held ? keys[i] : key_of((float)x[begin + i]);
  }
};

struct Cluster {
  cg::cluster_group group;
  Shared& sh;
  int rank, size;
  int shares, messages;  // exchanges so far: two buffers each, so that one barrier is enough
  // every block's share; returns the sums over all of them and over those in front of this one
  __device__ Share exchange(const Share& mine, Share& before) {
    Share* const buf = &sh.share[shares++ & 1];
    if (threadIdx.x == 0) *buf = mine;
    group.sync();
    Share all{0, 0, 0};
    before = all;
    for (int r = 0; r < size; ++r) {
      const Share s = *group.map_shared_rank(buf, r);
      if (r < rank) {
        before.sum += s.sum;
        before.count += s.count;
      }
      all.sum += s.sum;
      all.count += s.count;
      all.top = max(all.top, s.top);
    }
    return all;
  }
  // what the first block wrote to the message buffer
  __device__ Message* message() { return &sh.message[messages & 1]; }
  __device__ Message receive() {
    Message* const buf = message();
    ++messages;
    group.sync();
    return *group.map_shared_rank(buf, 0);
  }
};

// Counts (and weights) of the keys lo .. hi of the slice by class.  shift < 0: the first histogram.
template <class T>
__device__ void histogram(const Slice<T>& sl, const Scale& sc, Shared& sh, uint32_t lo, uint32_t hi, int shift,
                          bool weights) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins.n[i] = sh.bins.lo[i] = sh.bins.hi[i] = 0;
  __syncthreads();
  const int steps = (sl.n + kThreads - 1) / kThreads;
  for (int s = 0; s < steps; ++s) {
    const int i = s * kThreads + threadIdx.x;
    const uint32_t k = i < sl.n ? sl.key(i) : 0u;
    const bool in = k >= lo && k <= hi;
    const uint32_t lanes = __ballot_sync(0xffffffffu, in);
    if (!lanes) continue;
    const int b = !in ? 0 : shift < 0 ? bin_of(sc, k) : (int)((hi - k) >> shift);
    const uint64_t w = in && weights ? weight_of(sc, sh.table, k) : 0;
    // (equal logits, or a high temperature: a warp's elements in one class would queue up)
    const int b0 = __shfl_sync(0xffffffffu, b, __ffs(lanes) - 1);
    if (__all_sync(0xffffffffu, !in || b == b0)) {
      const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)w & 0x3FFFFFu),
                     high = __reduce_add_sync(0xffffffffu, (uint32_t)(w >> 22));
      if ((threadIdx.x & 31) == 0) {
        const uint64_t sum = ((uint64_t)high << 22) + low;
        atomicAdd(&sh.bins.n[b0], __popc(lanes));
        const uint32_t was = atomicAdd(&sh.bins.lo[b0], (uint32_t)sum);
        atomicAdd(&sh.bins.hi[b0], (uint32_t)(sum >> 32) + (was + (uint32_t)sum < was));
      }
    } else if (in) {
      atomicAdd(&sh.bins.n[b], 1u);
      if (w) {
        const uint32_t was = atomicAdd(&sh.bins.lo[b], (uint32_t)w), up = (uint32_t)(w >> 32) + (was + (uint32_t)w < was);
        if (up) atomicAdd(&sh.bins.hi[b], up);
      }
    }
  }
}

// What the first block knows of the search for a border.
struct Search {
  bool by_weight;     // the goal is a sum of weights (else a count)
  uint64_t goal;      // the border is the first token in the order with which the sum reaches it
  uint32_t lo, hi;    // keys of the classes of the last histogram
  int shift;          // -1: the first histogram
  uint32_t n_before;  // tokens and weights in front of them
  uint64_t w_before;
};

// Smallest or largest key of a class of the first histogram (a warp together): the classes rise as keys fall.
__device__ uint32_t first_key(const Scale& sc, int bin, bool largest) {
  // largest: the last key with bin_of >= bin, else the first with bin_of <= bin
  uint32_t lo = kLowestKey, hi = sc.top;
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 32 + 1;  // probes lo + step, lo + 2 step, ...
    const uint64_t at = (uint64_t)lo + (uint64_t)step * (lane + 1);
    const bool in = at <= hi;
    const int b = in ? bin_of(sc, (uint32_t)at) : 0;
    if (largest) {  // true for the keys up to the one sought
      const uint32_t yes = __ballot_sync(0xffffffffu, in && b >= bin);
      const int n = __popc(yes);
      hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)step * (n + 1) - 1);
      lo += step * n;
    } else {  // false for the keys in front of the one sought; the last key of the range is true
      const int b_lo = bin_of(sc, lo);
      if (b_lo <= bin) return lo;
      const uint32_t no = __ballot_sync(0xffffffffu, in && b > bin);
      const int n = __popc(no);
      hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)step * (n + 1));
      lo += step * n + 1;
    }
  }
  return lo;
}

// The first block: sums the cluster's histograms and keeps the running sums.
__device__ void merge(Cluster& cl, Shared& sh, uint32_t* cum_n, uint64_t* cum_w) {
  uint32_t n[kBinsPerThread];
  uint64_t w[kBinsPerThread];
  uint32_t tn = 0;
  uint64_t tw = 0;
#pragma unroll
  for (int q = 0; q < kBinsPerThread; ++q) n[q] = 0, w[q] = 0;
  for (int r = 0; r < cl.size; ++r) {
    const Shared* const o = cl.group.map_shared_rank(&sh, r);
#pragma unroll
    for (int q = 0; q < kBinsPerThread; ++q) {
      const int b = threadIdx.x * kBinsPerThread + q;
      n[q] += o->bins.n[b];
      w[q] += (uint64_t)o->bins.hi[b] << 32 | o->bins.lo[b];
    }
  }
#pragma unroll
  for (int q = 0; q < kBinsPerThread; ++q) {
    tn += n[q];
    tw += w[q];
  }
  block_scan(tn, tw, sh);
#pragma unroll
  for (int q = kBinsPerThread - 1; q >= 0; --q) {
    cum_n[threadIdx.x * kBinsPerThread + q] = tn;
    cum_w[threadIdx.x * kBinsPerThread + q] = tw;
    tn -= n[q];
    tw -= w[q];
  }
  __syncthreads();
}

// The first place of a rising array of running sums that reaches the goal (the block together).
template <class V>
__device__ int reaches(const V* cum, int n, uint64_t goal, Shared& sh) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (cum[i] >= goal && (i == 0 || cum[i - 1] < goal)) sh.bin = i;
  __syncthreads();
  const int b = sh.bin;
  __syncthreads();
  return b;
}

// The first block: what to do about the class that holds the border.
__device__ void next_step(Search& s, const Scale& sc, Shared& sh, Message* out) {
  const bool first = s.shift < 0;
  const uint32_t* const cum_n = first ? sh.first_n : sh.last_n;
  const uint64_t* const cum_w = first ? sh.first_w : sh.last_w;
  const int b = s.by_weight ? reaches(cum_w, kBins, s.goal - s.w_before, sh) : reaches(cum_n, kBins, s.goal - s.n_before, sh);
  const uint32_t upto = cum_n[b], in_front = b ? cum_n[b - 1] : 0u;
  const uint64_t w_front = b ? cum_w[b - 1] : 0;
  uint32_t lo, hi;
  if (first) {
    hi = first_key(sc, b, true);
    lo = first_key(sc, b, false);
  } else {
    hi = s.hi - ((uint32_t)b << s.shift);
    lo = max(s.lo, hi - ((1u << s.shift) - 1u));
  }
  Message m{};
  m.lo = lo;
  m.hi = hi;
  if (first && upto <= kList) {  // with all in front: a limit to the rest of top-k is among them, too
    m.op = kGather;
    m.hi = sc.top;
  } else {
    s.n_before += in_front;
    s.w_before += w_front;
    s.lo = lo;
    s.hi = hi;
    if (upto - in_front <= kList) {
      m.op = kGather;
    } else if (lo == hi) {
      m.op = kTies;
      const uint64_t w = weight_of(sc, sh.table, lo);
      m.border = s.by_weight ? (s.goal - s.w_before + w - 1) / w : s.goal - s.n_before;
    } else {
      m.op = kRefine;
      s.shift = max(0, 22 - __clz(hi - lo));
    }
  }
  if (threadIdx.x == 0) *out = m;
}

// Descending order of n entries (a power of two, at most kList), the block together
__device__ void sort_list(uint64_t* list, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const uint64_t x = list[a], y = list[b];
        if ((x < y) == ((a & size) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
}

// Sums of a slice by segment in the order of the index: f(key, index) gives what counts of an element.
// Afterwards `find` gives the index with which the sum over the row exceeds `target`.
template <class T, class F>
__device__ Share segments(const Slice<T>& sl, Shared& sh, Cluster& cl, Share& before, F f) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int len = ((sl.n + kSegs - 1) / kSegs + 31) & ~31;
  for (int s = wid; s < kSegs; s += kWarps) {
    uint64_t w = 0;
    uint32_t n = 0;
    const int end = min(sl.n, (s + 1) * len);
    for (int i = s * len; i < end; i += 32)
      if (i + lane < end) {
        uint64_t add = 0;
        if (f(sl.key(i + lane), sl.begin + i + lane, add)) ++n;
        w += add;
      }
    n = __reduce_add_sync(0xffffffffu, n);
    if (__any_sync(0xffffffffu, w != 0)) w = warp_sum(w);
    if (lane == 0) {
      sh.seg_sum[s] = w;
      sh.seg_n[s] = n;
    }
  }
  __syncthreads();
  if (wid == 0) {  // running sums over the segments
    uint64_t w = 0;
    uint32_t n = 0;
    for (int c = 0; c < kSegs; c += 32) {
      uint64_t x = sh.seg_sum[c + lane];
      n += __reduce_add_sync(0xffffffffu, sh.seg_n[c + lane]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x += w;
      sh.seg_sum[c + lane] = x;
      w = __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      sh.warp_w[0] = w;
      sh.warp_n[0] = n;
    }
  }
  __syncthreads();
  const Share all = cl.exchange(Share{sh.warp_w[0], sh.warp_n[0], 0}, before);
  return all;
}
// (the first warp of the block that holds it; else -1)
template <class T, class F>
__device__ int find(const Slice<T>& sl, Shared& sh, const Share& before, uint64_t target, F f) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x >= 32 || target < before.sum || target - before.sum >= sh.seg_sum[kSegs - 1]) return -1;
  const uint64_t rest = target - before.sum;
  int s = 0;
  for (int c = 0; c < kSegs; c += 32) s += __popc(__ballot_sync(0xffffffffu, sh.seg_sum[c + lane] <= rest));
  const int len = ((sl.n + kSegs - 1) / kSegs + 31) & ~31;
  uint64_t sum = s ? sh.seg_sum[s - 1] : 0;
  const int end = min(sl.n, (s + 1) * len);
  for (int i = s * len; i < end; i += 32) {
    uint64_t w = 0;
    if (i + lane < end) f(sl.key(i + lane), sl.begin + i + lane, w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, sum + w > rest);
    if (over) return i + __ffs(over) - 1;
    sum += __shfl_sync(0xffffffffu, w, 31);
  }
  return -1;
}

// The index of the m-th key (from 1) that equals k.
template <class T>
__device__ uint32_t tie(const Slice<T>& sl, Shared& sh, Cluster& cl, uint32_t k, uint64_t m) {
  auto equal = [&](uint32_t key, int, uint64_t& w) {
    w = key == k;
    return key == k;
  };
  Share before;
  segments(sl, sh, cl, before, equal);
  const int i = find(sl, sh, before, m - 1, equal);
  Share found{0, 0, 0};
  if (threadIdx.x == 0) sh.found = i >= 0 ? (uint32_t)(sl.begin + i) + 1u : 0u;
  __syncthreads();
  found.top = sh.found;
  Share unused;
  return cl.exchange(found, unused).top - 1u;
}

// 16 bytes of logits as values
__device__ __forceinline__ void values_of(const uint4& v, float (&x)[4], const float*) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
template <class H>
__device__ __forceinline__ void values_of(const uint4& v, float (&x)[8], const H*) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint16_t b = (uint16_t)((&v.x)[q >> 1] >> (16 * (q & 1)));
    x[q] = (float)*reinterpret_cast<const H*>(&b);
  }
}

// What the calls of a row have in common.
struct Row {
  float temperature, top_p, min_p, random;
  int top_k;
  __device__ bool fine() const {
    return temperature >= 0.f && temperature < INFINITY && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f &&
           min_p <= 1.f && random >= 0.f && random <= 1.f;
  }
};

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* const room = reinterpret_cast<uint32_t*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  Cluster cl{cg::this_cluster(), sh, 0, 0, 0, 0};
  cl.rank = (int)cl.group.block_rank();
  cl.size = (int)cl.group.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row = (int)(blockIdx.x / (unsigned)cl.size);
  Row r;
  r.temperature = p.temperature ? p.temperature[row] : 1.f;
  r.top_k = p.top_k ? p.top_k[row] : 0;
  r.top_p = p.top_p ? p.top_p[row] : 1.f;
  r.min_p = p.min_p ? p.min_p[row] : 0.f;
  r.random = p.random[row];

  // ---- the slice's keys to shared memory
  Slice<T> sl;
  sl.x = static_cast<const T*>(p.logits) + row * p.stride;
  sl.begin = min(p.vocab, cl.rank * p.slice);
  sl.n = min(p.vocab, sl.begin + p.slice) - sl.begin;
  constexpr int kVec = 16 / sizeof(T);
  // (keys stand as the logits do within 16 bytes, so that aligned loads become aligned stores)
  const T* const x0 = sl.x + sl.begin;
  const int skew = (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
  uint32_t* const keys = room + skew;
  sl.keys = keys;
  sl.held = min(sl.n, p.room);
  uint32_t top = 0, valid = 0;
  {
    const uint4* const base = reinterpret_cast<const uint4*>(x0 - skew);
    const int vecs = (skew + sl.n + kVec - 1) / kVec;
    constexpr int kAtOnce = 8;
    for (int v0 = tid; v0 < vecs; v0 += kThreads * kAtOnce) {
      uint4 v[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int j = v0 + q * kThreads, e = j * kVec - skew;  // first element
        v[q] = make_uint4(0u, 0u, 0u, 0u);
        if (e >= 0 && e + kVec <= sl.n) v[q] = __ldg(base + j);
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int j = v0 + q * kThreads, e = j * kVec - skew;
        if (j >= vecs) break;
        uint32_t k[kVec];
        if (e >= 0 && e + kVec <= sl.n) {
          float f[kVec];
          values_of(v[q], f, x0);
#pragma unroll
          for (int i = 0; i < kVec; ++i) k[i] = key_of(f[i]);
        } else {  // the slice's ends
#pragma unroll
          for (int i = 0; i < kVec; ++i) k[i] = e + i >= 0 && e + i < sl.n ? key_of((float)x0[e + i]) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          top = max(top, k[i]);
          valid += k[i] != 0u;
        }
        if (e >= 0 && e + kVec <= sl.held) {
#pragma unroll
          for (int i = 0; i < kVec; i += 4)
            *reinterpret_cast<uint4*>(keys + e + i) = make_uint4(k[i], k[i + 1], k[i + 2], k[i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (e + i >= 0 && e + i < sl.held) keys[e + i] = k[i];
        }
      }
    }
  }
  for (int i = tid; i < 1024; i += kThreads) sh.table[i] = __umul64hi(c_coarse[i >> 5], c_fine[i & 31]);
  top = __reduce_max_sync(0xffffffffu, top);
  valid = __reduce_add_sync(0xffffffffu, valid);
  if (lane == 0) {
    sh.warp_top[wid] = top;
    sh.warp_n[wid] = valid;
  }
  __syncthreads();
  top = valid = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    top = max(top, sh.warp_top[i]);
    valid += sh.warp_n[i];
  }
  Share before;
  const Share all = cl.exchange(Share{0, valid, top}, before);
  if (all.count == 0 || !r.fine()) {
    if (cl.rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.probs) p.probs[row] = 0.f;
      if (p.kept) p.kept[row] = 0;
    }
    cl.group.sync();  // a block's shared memory stays until the others have read it
    return;
  }

  // ---- the order's border: the last token that top-k and top-p keep
  const bool greedy = r.temperature == 0.f;
  const Scale sc = scale_of(all.top, greedy ? 1.f : r.temperature);
  uint64_t border = 0;
  if (greedy) {
    border = order_of(all.top, tie(sl, sh, cl, all.top, 1));
  } else {
    const bool by_count = r.top_k > 0 && (uint32_t)r.top_k < all.count, by_weight = r.top_p < 1.f;
    if (by_count || by_weight) {
      histogram(sl, sc, sh, 1u, 0xFFFFFFFFu, -1, by_weight);
      cl.group.sync();
      Search se{};  // (of use in the first block)
      // the weight that top-p of a sum of w asks for
      auto part_of = [&](uint64_t w) {
        return max((uint64_t)1, min(w, (uint64_t)__double2ull_ru((double)r.top_p * (double)w)));
      };
      auto restart = [&](uint64_t whole) {  // top-p of what top-k keeps, from the first histogram on
        se.by_weight = true;
        se.goal = part_of(whole);
        se.shift = -1;
        se.n_before = 0;
        se.w_before = 0;
      };
      if (cl.rank == 0) {
        merge(cl, sh, sh.first_n, sh.first_w);
        se.shift = -1;
        if (by_count) {
          se.goal = (uint64_t)r.top_k;
        } else {
          restart(sh.first_w[kBins - 1]);
        }
        sh.n_list = 0;
        next_step(se, sc, sh, cl.message());
      }
      for (;;) {
        const Message m = cl.receive();
        if (m.op == kDone) {
          border = m.border;
          break;
        }
        if (m.op == kGather) {
          Shared* const to = cl.group.map_shared_rank(&sh, 0);
          const int steps = (sl.n + kThreads - 1) / kThreads;
          for (int s = 0; s < steps; ++s) {
            const int i = s * kThreads + tid;
            const uint32_t k = i < sl.n ? sl.key(i) : 0u;
            if (k >= m.lo && k <= m.hi) {
              const uint32_t at = atomicAdd(&to->n_list, 1u);
              if (at < kList) to->list[at] = order_of(k, (uint32_t)(sl.begin + i));
            }
          }
          cl.group.sync();
          if (cl.rank == 0) {
            const int n = (int)min(sh.n_list, (uint32_t)kList);
            int size = 32;
            while (size < n) size <<= 1;
            for (int i = n + tid; i < size; i += kThreads) sh.list[i] = 0;
            __syncthreads();
            sort_list(sh.list, size);
            // running sums of the weights
            uint64_t w[kBinsPerThread], sum = 0;
            uint32_t none = 0;
#pragma unroll
            for (int q = 0; q < kBinsPerThread; ++q) {
              const int i = tid * kBinsPerThread + q;
              w[q] = by_weight && i < n ? weight_of(sc, sh.table, (uint32_t)(sh.list[i] >> 32)) : 0;
              sum += w[q];
            }
            block_scan(none, sum, sh);
#pragma unroll
            for (int q = kBinsPerThread - 1; q >= 0; --q) {
              sh.last_w[tid * kBinsPerThread + q] = sum;
              sum -= w[q];
            }
            __syncthreads();
            int at = se.by_weight ? reaches(sh.last_w, n, se.goal - se.w_before, sh) : (int)(se.goal - se.n_before) - 1;
            bool done = true;
            if (!se.by_weight && by_weight) {
              const uint64_t w_front = se.w_before;
              restart(w_front + sh.last_w[at]);
              done = se.goal > w_front;  // (else in front of these)
              if (done) at = reaches(sh.last_w, n, se.goal - w_front, sh);
            }
            if (done) {
              if (tid == 0) *cl.message() = Message{kDone, 0, 0, sh.list[at]};
            } else {
              if (tid == 0) sh.n_list = 0;
              next_step(se, sc, sh, cl.message());
            }
          }
        } else if (m.op == kRefine) {
          const int shift = max(0, 22 - __clz(m.hi - m.lo));
          histogram(sl, sc, sh, m.lo, m.hi, shift, by_weight);
          cl.group.sync();
          if (cl.rank == 0) {
            merge(cl, sh, sh.last_n, sh.last_w);
            next_step(se, sc, sh, cl.message());
          }
        } else {
          const uint32_t index = tie(sl, sh, cl, m.lo, m.border);
          if (cl.rank == 0) {
            bool done = true;
            if (!se.by_weight && by_weight) {
              const uint64_t w = weight_of(sc, sh.table, m.lo), w_front = se.w_before;
              restart(w_front + m.border * w);
              done = se.goal > w_front;
              if (done && tid == 0) *cl.message() = Message{kTies, m.lo, m.lo, (se.goal - w_front + w - 1) / w};
            } else if (tid == 0) {
              *cl.message() = Message{kDone, 0, 0, order_of(m.lo, index)};
            }
            if (!done) next_step(se, sc, sh, cl.message());
          }
        }
      }
    }
  }

  // ---- the draw among the tokens up to the border, and with min-p's weight
  const uint64_t least = greedy ? 0 : (uint64_t)__double2ull_ru((double)r.min_p * (double)(1ull << kOneBits));
  auto kept = [&](uint32_t key, int index, uint64_t& w) {
    if (key == 0u || order_of(key, (uint32_t)index) < border) return false;
    w = weight_of(sc, sh.table, key);
    if (w >= least) return true;
    w = 0;
    return false;
  };
  const Share sum = segments(sl, sh, cl, before, kept);
  const uint64_t target = min(sum.sum - 1, (uint64_t)((double)r.random * (double)sum.sum));
  const int i = find(sl, sh, before, target, kept);
  if (i >= 0 && lane == 0) {
    p.tokens[row] = sl.begin + i;
    if (p.kept) p.kept[row] = (int32_t)sum.count;
    if (p.probs) {
      // (the weight as a number: its multiple of 2^-42 may have few bits)
      const uint32_t k = sl.key(i);
      float h = 0.f, l = 0.f;
      if (k != sc.top) log2_below(sc, k, h, l);
      p.probs[row] = (float)((double)(exp2f(-h) * (1.f - 0.6931471805599453f * l)) * (double)(1ull << kOneBits) / (double)sum.sum);
    }
  }
  cl.group.sync();  // a block's shared memory stays until the others have read it
}

template <class T>
cudaError_t launch(SampleArgs p, int sms, int most_smem, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit for this kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // Blocks per row: more of them while the rows alone leave SMs idle or a slice is so large that only one
  // block fits an SM; a slice has at least 2,048 logits (a cluster's barriers cost what its blocks save).
  constexpr int kTwoPerSm = 16384, kLeast = 2048;
  int blocks = 1;
  while (blocks < kMaxCluster && p.vocab / blocks >= 2 * kLeast &&
         ((int64_t)p.n_rows * blocks < sms || (p.vocab - 1) / blocks + 1 > kTwoPerSm))
    blocks *= 2;
  p.slice = (p.vocab - 1) / blocks + 1;
  const int fixed = (int)(sizeof(Shared) + 15) / 16 * 16 + 64;
  p.room = std::min(p.slice, (most_smem - fixed) / 4);
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)p.n_rows * blocks);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = fixed + 4 * (size_t)p.room;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, sample_kernel<T>, p);
}
}  // namespace

cudaError_t launch_sample(const SampleArgs& p, int dtype, int sms, cudaStream_t s) {
  constexpr int kSmem = 227 * 1024;
  if (dtype == MSM_FP32) return launch<float>(p, sms, kSmem, s);
  return dtype == MSM_BF16 ? launch<__nv_bfloat16>(p, sms, kSmem, s) : launch<__half>(p, sms, kSmem, s);
}

}  // namespace msm
