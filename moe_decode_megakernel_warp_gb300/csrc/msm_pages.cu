// msm_pages.cu — the page operations of a paged KV cache: reserving and freeing pages
// (with a copy of a shared last page), sharing them between sequences, moving the pages
// in use to the front of the pool, and storing new K/V rows.
//
// The bookkeeping of one call runs in one thread-block cluster: its phases (check,
// count, assign) need the whole cache's totals between them, which the blocks exchange
// through distributed shared memory and cluster barriers inside one launch.  Page
// indices are given out by rank (the k-th missing page is the k-th lowest free one,
// both counted by prefix sums), so the result does not depend on the order of threads.
// The rows that a call moves are copied by a second launch over the whole GPU, chained
// with programmatic dependent launch; it reads the list that the first one left.
#include <cooperative_groups.h>

#include <algorithm>

#include "msm_device.cuh"
#include "msm_paged.h"

namespace cg = cooperative_groups;

namespace msm {
namespace {

// Threads per block (N below): 1,024, or 256 where the eight blocks' 64 warps have a sequence each
// at most and 16,384 pages are one look: their barriers cost less (a resize of 32 sequences 8.6
// -> 7.4 us, a compaction of 150 pages 8.8 -> 7.8), and only larger caches miss the others (a fork
// of 64 sequences into 256: 7.0 us with 1,024, 9.0 with 256).
constexpr int kMetaMost = 1024, kMetaFew = 256;
constexpr int kMetaBlocks = 8;      // the portable cluster size
constexpr int kPagesPerThread = 8;  // pages one thread looks at per step of a scan

// a resize or fork that is not done: the calls behind it change nothing either
__device__ __forceinline__ void refuse(int32_t* status, int code, int call) {
  latch(status, code, call);
  atomicOr(status, kPagesStopped);
}

struct BlockShare {        // what a block tells the others
  int need, count, holes;  // missing pages, free (or live) pages, holes below the live count
  int bad;
};

struct Share {
  BlockShare mine;
  BlockShare all[kMetaBlocks];
  int warp_sum[kMetaMost / 32];
};

// exclusive prefix of x over the block's threads; total = the block's sum
template <int N>
__device__ int block_scan(int x, Share& sh, int& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sh.warp_sum[wid] = v;
  __syncthreads();
  int w = lane < N / 32 ? sh.warp_sum[lane] : 0, t = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  total = __shfl_sync(0xffffffffu, t, 31);
  const int before = __shfl_sync(0xffffffffu, t - w, wid);
  __syncthreads();  // warp_sum may be written again
  return before + v - x;
}

// every block's share, visible to all of them after this barrier
__device__ void exchange(Share& sh, cg::cluster_group& cl) {
  cl.sync();
  if (threadIdx.x < kMetaBlocks) sh.all[threadIdx.x] = *cl.map_shared_rank(&sh.mine, threadIdx.x);
  __syncthreads();
}

// the block's share of n things
__device__ __forceinline__ void block_range(int n, int rank, int& lo, int& hi) {
  const int per = (n - 1) / kMetaBlocks + 1;
  lo = (int)min((int64_t)n, (int64_t)rank * per);
  hi = min(n, lo + per);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// pages of [lo, hi) that are free (live = false) or in use
template <int N>
__device__ int count_pages(const int32_t* refs, int lo, int hi, bool live, Share& sh) {
  int n = 0;
  for (int p = lo + (int)threadIdx.x; p < hi; p += N * kPagesPerThread) {
    int r[kPagesPerThread];
#pragma unroll
    for (int q = 0; q < kPagesPerThread; ++q) {
      const int i = p + q * N;
      r[q] = i < hi ? __ldcg(refs + i) : (live ? 0 : 1);
    }
#pragma unroll
    for (int q = 0; q < kPagesPerThread; ++q) n += (r[q] > 0) == live;
  }
  int total;
  block_scan<N>(n, sh, total);
  return total;
}

template <int N>
__global__ void __cluster_dims__(kMetaBlocks, 1, 1) __launch_bounds__(N)
    resize_kernel(const PagesMeta p) {
  __shared__ Share sh;
  pdl_launch_dependents();  // the copy launch waits for this one's end itself
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const PagesScratch sc(p.scratch, p.n_pages, p.n_seqs);
  const int64_t cap = (int64_t)p.max_pages * p.page_rows;
  int s0, s1, p0, p1;
  block_range(p.n_seqs, rank, s0, s1);
  block_range(p.n_pages, rank, p0, p1);
  if (threadIdx.x == 0) sh.mine.bad = 0;
  if (rank == 0 && threadIdx.x == 0) sc.head[0] = 0;
  const bool stop = stopped(p.status);
  __syncthreads();

  // free pages among this thread's first kPagesPerThread of the block's share (their loads
  // travel during step 1)
  const int mine = p0 + (int)threadIdx.x * kPagesPerThread;
  uint32_t mine_free = 0;
#pragma unroll
  for (int q = 0; q < kPagesPerThread; ++q)
    if (mine + q < p1 && __ldcg(p.refs + mine + q) <= 0) mine_free |= 1u << q;
  const int p_rest = p0 + N * kPagesPerThread;  // the share's pages behind those

  // 1. each sequence: are its lengths and the pages it gives up in range, how many pages
  //    does it lack, does it have to leave a shared last page (offset = 2 pages + leave, unsigned:
  //    the sequences' needs add up to fewer than 2^31 pages, a table's entries)
  for (int s = s0 + wid; s < s1; s += (N / 32)) {
    const int old = p.lens[s], asked = p.arg[s], now = asked == -1 ? old : asked;
    bool bad = old < 0 || old > cap || now < 0 || now > cap;
    int need = 0, leave = 0;
    if (!bad) {
      const int32_t* row = p.table + (size_t)s * p.max_pages;
      const int n_old = ceil_div(old, p.page_rows), n_new = ceil_div(now, p.page_rows);
      for (int j = n_new + lane; j < n_old; j += 32) {
        const int pg = row[j];
        bad |= pg < 0 || pg >= p.n_pages || p.refs[pg] <= 0;
      }
      if (now > old && old % p.page_rows) {
        const int pg = row[old / p.page_rows];
        bad |= pg < 0 || pg >= p.n_pages;
        if (!bad) leave = p.refs[pg] > 1;
      }
      need = max(0, n_new - n_old) + leave;
    }
    if (__any_sync(0xffffffffu, bad)) {
      sh.mine.bad = 1;
      need = leave = 0;
    }
    if (lane == 0) sc.offset[s] = (int32_t)(2u * (uint32_t)need + (uint32_t)leave);
  }
  __syncthreads();
  // 2. prefix of the needs over the block's sequences, free pages of its share of the pool
  int base = 0;
  for (int c = s0; c < s1; c += N) {
    const int s = c + (int)threadIdx.x;
    const uint32_t e = s < s1 ? (uint32_t)sc.offset[s] : 0u;
    int total;
    const int before = block_scan<N>((int)(e >> 1), sh, total);
    if (s < s1) sc.offset[s] = (int32_t)(2u * (uint32_t)(base + before) + (e & 1u));
    base += total;
  }
  int n_free;
  const int mine_rank = block_scan<N>(__popc(mine_free), sh, n_free);
  if (p_rest < p1) n_free += count_pages<N>(p.refs, p_rest, p1, false, sh);
  if (threadIdx.x == 0) {
    sh.mine.need = base;
    sh.mine.count = n_free;
  }
  exchange(sh, cl);
  int need_before = 0, free_before = 0, bad = 0;
  int64_t need_all = 0, free_all = 0;
#pragma unroll
  for (int b = 0; b < kMetaBlocks; ++b) {
    if (b < rank) {
      need_before += sh.all[b].need;
      free_before += sh.all[b].count;
    }
    need_all += sh.all[b].need;
    free_all += sh.all[b].count;
    bad |= sh.all[b].bad;
  }
  if (stop || bad || need_all > free_all) {
    if (!stop && rank == 0 && threadIdx.x == 0) refuse(p.status, bad ? MSM_ERR_INVALID_ARG : MSM_ERR_OOM, kCallResize);
    cl.sync();  // a block's shared memory stays until the others have read it
    return;
  }
  // 3. list[r] = the r-th lowest free page, for the r that are needed
  auto give = [&](int first, uint32_t mask, int64_t r) {
#pragma unroll
    for (int q = 0; q < kPagesPerThread; ++q)
      if (mask >> q & 1) {
        if (r < need_all) sc.list[r] = first + q;
        ++r;
      }
  };
  if (free_before < need_all) {
    give(mine, mine_free, (int64_t)free_before + mine_rank);
    int64_t at = free_before;
    if (p_rest < p1) {
      int first_step;
      block_scan<N>(__popc(mine_free), sh, first_step);
      at += first_step;
    }
    for (int c = p_rest; c < p1 && at < need_all; c += N * kPagesPerThread) {
      const int q0 = c + (int)threadIdx.x * kPagesPerThread;
      uint32_t mask = 0;
#pragma unroll
      for (int q = 0; q < kPagesPerThread; ++q)
        if (q0 + q < p1 && __ldcg(p.refs + q0 + q) <= 0) mask |= 1u << q;
      int total;
      const int before = block_scan<N>(__popc(mask), sh, total);
      give(q0, mask, at + before);
      at += total;
    }
  }
  cl.sync();
  // 4. the tables
  for (int s = s0 + wid; s < s1; s += (N / 32)) {
    const int old = p.lens[s], asked = p.arg[s], now = asked == -1 ? old : asked;
    if (now == old) continue;
    int32_t* row = p.table + (size_t)s * p.max_pages;
    const int n_old = ceil_div(old, p.page_rows), n_new = ceil_div(now, p.page_rows);
    const uint32_t e = (uint32_t)sc.offset[s];
    int off = need_before + (int)(e >> 1);
    if (e & 1u) {
      if (lane == 0) {
        const int j = old / p.page_rows, from = row[j], to = __ldcg(sc.list + off);
        const int i = atomicAdd(sc.head, 1);
        sc.copies[3 * i] = from;
        sc.copies[3 * i + 1] = to;
        sc.copies[3 * i + 2] = old % p.page_rows;
        row[j] = to;
        p.refs[to] = 1;
        atomicSub(p.refs + from, 1);
      }
      ++off;
    }
    for (int j = n_old + lane; j < n_new; j += 32) {
      const int pg = __ldcg(sc.list + off + j - n_old);
      row[j] = pg;
      p.refs[pg] = 1;
    }
    for (int j = n_new + lane; j < n_old; j += 32) {
      atomicSub(p.refs + row[j], 1);
      row[j] = -1;
    }
    if (lane == 0) p.lens[s] = now;
  }
}

template <int N>
__global__ void __cluster_dims__(kMetaBlocks, 1, 1) __launch_bounds__(N)
    fork_kernel(const PagesMeta p) {
  __shared__ Share sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t cap = (int64_t)p.max_pages * p.page_rows;
  const int w0 = rank * (N / 32) + wid, n_warps = kMetaBlocks * (N / 32);
  const bool stop = stopped(p.status);
  if (threadIdx.x == 0) sh.mine.bad = 0;
  __syncthreads();
  for (int s = w0; s < p.n_seqs; s += n_warps) {
    const int par = p.arg[s];
    if (par == -1) continue;
    bool bad = par < 0 || par >= p.n_seqs || par == s || p.lens[s] != 0;
    if (!bad) {
      const int len = p.lens[par];
      bad = p.arg[par] != -1 || len < 0 || len > cap;
      if (!bad)
        for (int j = lane; j < ceil_div(len, p.page_rows); j += 32) {
          const int pg = p.table[(size_t)par * p.max_pages + j];
          bad |= pg < 0 || pg >= p.n_pages || p.refs[pg] <= 0;
        }
    }
    if (__any_sync(0xffffffffu, bad)) sh.mine.bad = 1;
  }
  exchange(sh, cl);
  int bad = 0;
#pragma unroll
  for (int b = 0; b < kMetaBlocks; ++b) bad |= sh.all[b].bad;
  cl.sync();
  if (stop || bad) {
    if (!stop && rank == 0 && threadIdx.x == 0) refuse(p.status, MSM_ERR_INVALID_ARG, kCallFork);
    return;
  }
  for (int s = w0; s < p.n_seqs; s += n_warps) {
    const int par = p.arg[s];
    if (par == -1) continue;
    const int len = p.lens[par];
    for (int j = lane; j < ceil_div(len, p.page_rows); j += 32) {
      const int pg = p.table[(size_t)par * p.max_pages + j];
      p.table[(size_t)s * p.max_pages + j] = pg;
      atomicAdd(p.refs + pg, 1);
    }
    if (lane == 0) p.lens[s] = len;
  }
}

// With L pages in use, the moves pair the free indices below L with the pages in use at
// L and above, both ascending.  A page in use with `before` of them in front of it is the
// (L - 1 - before)-th from the end, so the sources are listed from their end, which needs
// no count of the pages in use below L; the destinations are listed from the front.
template <int N>
__global__ void __cluster_dims__(kMetaBlocks, 1, 1) __launch_bounds__(N)
    compact_kernel(const PagesMeta p) {
  __shared__ Share sh;
  pdl_launch_dependents();  // the copy launch waits for this one's end itself
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const PagesScratch sc(p.scratch, p.n_pages, p.n_seqs);
  int32_t* const dst = sc.list + p.n_pages / 2;
  int p0, p1;
  block_range(p.n_pages, rank, p0, p1);
  const bool stop = stopped(p.status);
  const int n_live = count_pages<N>(p.refs, p0, p1, true, sh);
  if (threadIdx.x == 0) {
    sh.mine.count = n_live;
    sh.mine.holes = 0;
  }
  exchange(sh, cl);
  int at = 0, live = 0;
#pragma unroll
  for (int b = 0; b < kMetaBlocks; ++b) {
    if (b < rank) at += sh.all[b].count;
    live += sh.all[b].count;
  }
  int holes = 0;
  for (int c = p0; c < p1; c += N * kPagesPerThread) {
    const int q0 = c + (int)threadIdx.x * kPagesPerThread;
    uint32_t mask = 0;
#pragma unroll
    for (int q = 0; q < kPagesPerThread; ++q)
      if (q0 + q < p1 && __ldcg(p.refs + q0 + q) > 0) mask |= 1u << q;
    int total;
    int before = at + block_scan<N>(__popc(mask), sh, total);
#pragma unroll
    for (int q = 0; q < kPagesPerThread; ++q) {
      const int pg = q0 + q;
      if (pg >= p1) break;
      const bool used = mask >> q & 1;
      if (pg >= live) {
        sc.to[pg] = pg;
        if (used) sc.list[live - 1 - before] = pg;
      } else if (!used) {
        dst[pg - before] = pg;
        ++holes;
      }
      before += used;
    }
    at += total;
  }
  int block_holes;
  block_scan<N>(holes, sh, block_holes);
  if (threadIdx.x == 0) sh.mine.holes = block_holes;
  exchange(sh, cl);
  int moves = 0;
#pragma unroll
  for (int b = 0; b < kMetaBlocks; ++b) moves += stop ? 0 : sh.all[b].holes;
  for (int m = rank * N + (int)threadIdx.x; m < moves; m += kMetaBlocks * N) {
    const int from = __ldcg(sc.list + moves - 1 - m), to = __ldcg(dst + m);
    sc.to[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    sc.head[0] = moves;
    sc.head[1] = stop ? p.n_pages : live;  // pages from here on are renumbered
  }
  cl.sync();  // a block's shared memory stays until the others have read it
}

// ---------------------------------------------------------------- row copies
// Bound by memory: each byte is read once and written once.  blockIdx.y = (layer, K or V); the
// warps of a row of blocks share out the pieces of up to 8 KB, 16 loads of 16 bytes in flight
// per lane (8: 20 % slower on short runs).  The scales of a cache in 8 bits are behind its rows in
// blockIdx.y, an entry per warp.
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 16;  // 16-byte vectors per lane
constexpr int kPieceVecs = 32 * kCopyVecs;

template <bool kCompact>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PagesCopy p) {
  pdl_wait();
  const PagesScratch sc(p.m.scratch, p.m.n_pages, p.m.n_seqs);
  const int32_t* const dst = sc.list + p.m.n_pages / 2;
  const int lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * kCopyThreads + threadIdx.x) >> 5, warps = (gridDim.x * kCopyThreads) >> 5;
  const uint32_t entries = sc.head[0];
  if ((int)blockIdx.y >= 2 * p.n_layers) {
    const int layer = (blockIdx.y >> 1) - p.n_layers;
    float* const scales = blockIdx.y & 1 ? p.v_scales[layer] : p.k_scales[layer];
    const int64_t page_scales = (int64_t)p.n_kv_heads * p.page_blocks;
    for (uint32_t e = warp; e < entries; e += warps) {
      const int from = kCompact ? sc.list[entries - 1 - e] : sc.copies[3 * (size_t)e];
      const int to = kCompact ? dst[e] : sc.copies[3 * (size_t)e + 1];
      // those of the rows that are copied
      const int blocks = kCompact ? p.page_blocks : ceil_div(sc.copies[3 * (size_t)e + 2], p.block_rows);
      for (int64_t i = lane; i < (int64_t)p.n_kv_heads * blocks; i += 32) {
        const int64_t at = i / blocks * p.page_blocks + i % blocks;
        scales[to * page_scales + at] = scales[from * page_scales + at];
      }
    }
    return;
  }
  // a page is n_kv_heads runs of page_rows rows; all of it is one run when it moves whole
  const int64_t head_vecs = (int64_t)p.m.page_rows * p.row_vecs, page_vecs = head_vecs * p.n_kv_heads;
  const int64_t run_vecs = kCompact ? page_vecs : head_vecs;
  const uint32_t pieces = (uint32_t)((run_vecs + kPieceVecs - 1) / kPieceVecs);
  const uint32_t per_entry = kCompact ? pieces : pieces * p.n_kv_heads;
  uint4* const pool = blockIdx.y & 1 ? p.v[blockIdx.y >> 1] : p.k[blockIdx.y >> 1];
  for (uint64_t u = warp; u < (uint64_t)entries * per_entry; u += warps) {
    // (a pool holds fewer than 2^32 rows, so fewer than 2^32 pieces)
    const uint32_t e = (uint32_t)u / per_entry, r = (uint32_t)u - e * per_entry;
    const uint32_t run = kCompact ? 0 : r / pieces;
    const int64_t first = (int64_t)(r - run * pieces) * kPieceVecs;
    int from, to;
    int64_t n = run_vecs;
    if (kCompact) {
      from = sc.list[entries - 1 - e];
      to = dst[e];
    } else {
      from = sc.copies[3 * (size_t)e];
      to = sc.copies[3 * (size_t)e + 1];
      n = (int64_t)sc.copies[3 * (size_t)e + 2] * p.row_vecs;
    }
    if (first >= n) continue;
    const uint4* const src = pool + from * page_vecs + run * run_vecs + first;
    uint4* const out = pool + to * page_vecs + run * run_vecs + first;
    const int left = (int)min(n - first, (int64_t)kPieceVecs);
    uint4 x[kCopyVecs];
#pragma unroll
    for (int q = 0; q < kCopyVecs; ++q)
      if (q * 32 + lane < left) x[q] = __ldcs(src + q * 32 + lane);
#pragma unroll
    for (int q = 0; q < kCopyVecs; ++q)
      if (q * 32 + lane < left) __stcs(out + q * 32 + lane, x[q]);
  }
  if (kCompact && p.renumber && blockIdx.y == 0) {
    const int live = sc.head[1];
    for (int64_t s = warp; s < p.m.n_seqs; s += warps) {
      const int n = ceil_div(min(max(p.m.lens[s], 0), p.m.max_pages * p.m.page_rows), p.m.page_rows);
      int32_t* const row = p.m.table + s * p.m.max_pages;
      for (int j = lane; j < n; j += 32) {
        const int pg = row[j];
        if (pg >= live && pg < p.m.n_pages) row[j] = sc.to[pg];
      }
    }
  }
}

// ---------------------------------------------------------------- new rows
// Bound by memory (and by latency for a step's few tokens): one warp per token.  Its loads
// do not depend on where the rows go, so they are on their way while the warp looks that up.
constexpr int kWriteThreads = 128;
constexpr int kWriteVecs = 8;  // 16-byte vectors per lane at a time

__global__ void __launch_bounds__(kWriteThreads) write_kernel(const PagesWrite p) {
  const int lane = threadIdx.x & 31;
  const int t = (int)((blockIdx.x * (int64_t)kWriteThreads + threadIdx.x) >> 5);
  if (t >= p.n_tokens || t >= p.starts[p.m.n_seqs]) return;
  const bool stop = stopped(p.m.status);
  const int half = p.n_kv_heads << p.row_shift, n = 2 * half;
  auto load = [&](int i) -> uint4 {
    const bool v = i >= half;
    const int r = v ? i - half : i, h = r >> p.row_shift, c = r & ((1 << p.row_shift) - 1);
    return v ? __ldcs(p.v + t * p.v_token + h * p.v_head + c) : __ldcs(p.k + t * p.k_token + h * p.k_head + c);
  };
  uint4 x[kWriteVecs];
#pragma unroll
  for (int q = 0; q < kWriteVecs; ++q)
    if (lane + q * 32 < n) x[q] = load(lane + q * 32);
  // the last sequence that starts at or before the token, 32 probes at a time
  int lo = 0, hi = p.m.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, i < hi && p.starts[i] <= t);
    lo += le ? (31 - __clz(le)) * step : 0;
    hi = min(hi, lo + step);
  }
  const int first = p.starts[lo], end = p.starts[lo + 1];
  const int64_t pos = (int64_t)p.m.lens[lo] - end + t;
  bool ok = t >= first && t < end && pos >= 0 && pos < (int64_t)p.m.max_pages * p.m.page_rows;
  int64_t at = 0;  // pool vector of head 0 of the token's row
  if (ok) {
    const int pg = p.m.table[(size_t)lo * p.m.max_pages + (int)pos / p.m.page_rows];
    ok = pg >= 0 && pg < p.m.n_pages && p.m.refs[pg] == 1;
    at = ((int64_t)pg * p.n_kv_heads * p.m.page_rows + (int)pos % p.m.page_rows) << p.row_shift;
  }
  if (!ok || stop) {
    if (lane == 0 && !stop) latch(p.m.status, MSM_ERR_INVALID_ARG, kCallWrite);
    return;
  }
  const int64_t head = (int64_t)p.m.page_rows << p.row_shift;
  for (int i0 = lane; i0 < n; i0 += 32 * kWriteVecs) {
    if (i0 != lane) {
#pragma unroll
      for (int q = 0; q < kWriteVecs; ++q)
        if (i0 + q * 32 < n) x[q] = load(i0 + q * 32);
    }
#pragma unroll
    for (int q = 0; q < kWriteVecs; ++q) {
      const int i = i0 + q * 32;
      if (i >= n) break;
      const bool v = i >= half;
      const int r = v ? i - half : i, h = r >> p.row_shift, c = r & ((1 << p.row_shift) - 1);
      (v ? p.pool_v : p.pool_k)[at + h * head + c] = x[q];
    }
  }
}

}  // namespace

namespace {
bool few(const PagesMeta& p) {
  return p.n_seqs <= kMetaBlocks * kMetaFew / 32 && p.n_pages <= kMetaBlocks * kMetaFew * kPagesPerThread;
}
}  // namespace

cudaError_t launch_pages_resize(const PagesMeta& p, cudaStream_t s) {
  if (few(p)) resize_kernel<kMetaFew><<<kMetaBlocks, kMetaFew, 0, s>>>(p);
  else resize_kernel<kMetaMost><<<kMetaBlocks, kMetaMost, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesMeta& p, cudaStream_t s) {
  if (few(p)) fork_kernel<kMetaFew><<<kMetaBlocks, kMetaFew, 0, s>>>(p);
  else fork_kernel<kMetaMost><<<kMetaBlocks, kMetaMost, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesMeta& p, cudaStream_t s) {
  if (few(p)) compact_kernel<kMetaFew><<<kMetaBlocks, kMetaFew, 0, s>>>(p);
  else compact_kernel<kMetaMost><<<kMetaBlocks, kMetaMost, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PagesCopy& p, bool compact, int sms, cudaStream_t s) {
  // at most as many warps as there can be pieces, about sixteen blocks per SM in all
  const int64_t vecs = (int64_t)p.m.page_rows * p.row_vecs * (compact ? p.n_kv_heads : 1);
  const int64_t pieces = (vecs - 1) / kPieceVecs + 1;
  const int64_t entries = compact ? p.m.n_pages / 2 : p.m.n_seqs;
  const int64_t warps = entries * pieces * (compact ? 1 : p.n_kv_heads);
  const int ys = 2 * p.n_layers * (p.page_blocks ? 2 : 1);
  const int64_t blocks = (warps - 1) / (kCopyThreads / 32) + 1, most = (16 * sms - 1) / (2 * p.n_layers) + 1;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min(blocks, most)), ys);
  lc.blockDim = dim3(kCopyThreads);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return compact ? cudaLaunchKernelEx(&lc, copy_kernel<true>, p) : cudaLaunchKernelEx(&lc, copy_kernel<false>, p);
}

cudaError_t launch_pages_write(const PagesWrite& p, cudaStream_t s) {
  constexpr int kTokens = kWriteThreads / 32;
  write_kernel<<<(p.n_tokens - 1) / kTokens + 1, kWriteThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace msm
