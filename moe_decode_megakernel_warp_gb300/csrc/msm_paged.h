// Launch interfaces of the paged-cache kernels (msm_pages.cu), shared with the host
// side (msm_paged_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "msm.h"

namespace msm {

// sets the calling thread's error message (msm_last_error) and returns `st`
msm_status report(msm_status st, const char* msg);
msm_status report_cuda(cudaError_t e, const char* what);

// device status word of a cache: the msm_status of the first error in the low byte, its call in the
// next one, and whether a resize or fork was refused.  From then on, until msm_pages_sync clears the
// word, no call changes the cache: the lengths are not those that the following calls
// count on (a write would store its rows over the last ones of the history).
enum PagesCall { kCallResize = 1, kCallFork = 2, kCallWrite = 3, kCallAttention = 4 };
constexpr int kPagesStopped = 1 << 16;

// scratch of a cache: counters, one offset per sequence, a list of row copies (source
// page, destination page, rows) per sequence, and two page-sized arrays
constexpr int kScratchHead = 16;
struct PagesScratch {
  int32_t *head, *offset, *copies, *list, *to;
  __host__ __device__ PagesScratch(int32_t* base, int n_pages, int n_seqs)
      : head(base),
        offset(base + kScratchHead),
        copies(offset + n_seqs),
        list(copies + 3 * (size_t)n_seqs),
        to(list + n_pages) {}
};
inline size_t pages_scratch_ints(int n_pages, int n_seqs) {
  return kScratchHead + 4 * (size_t)n_seqs + 2 * (size_t)n_pages;
}

struct PagesMeta {
  int32_t *table, *lens, *refs, *status, *scratch;
  const int32_t* arg;  // new_lens or parent
  int n_pages, page_rows, n_seqs, max_pages;
};

constexpr int kPagesLayers = 64;  // layers of one copy launch (their pool pointers travel as parameters)
struct PagesCopy {
  PagesMeta m;
  int n_layers, n_kv_heads, row_vecs;  // 16-byte vectors per row
  int renumber;                        // compact: this launch also renumbers the tables
  int block_rows, page_blocks;         // a cache in 8 bits: rows of a scale, scales of a page and head (else 0)
  uint4* k[kPagesLayers];
  uint4* v[kPagesLayers];
  float* k_scales[kPagesLayers];
  float* v_scales[kPagesLayers];
};

struct PagesWrite {
  PagesMeta m;
  int n_kv_heads, row_shift, n_tokens;  // 2^row_shift 16-byte vectors per row
  uint4 *pool_k, *pool_v;
  const uint4 *k, *v;
  int64_t k_token, k_head, v_token, v_head;  // strides in 16-byte vectors
  const int32_t* starts;
};

// Division of 0 .. 2^31 - 1 by a number that a launch knows: with 2^l the least power of two that is not below d,
// m = ceil(2^(31 + l) / d) is below 2^32 and exceeds the quotient by less than 2^l / 2^(31 + l) of it, so the
// product's upper part is the quotient's integer.
struct Divisor {
  uint32_t d, mul, shift;
  explicit Divisor(int by = 1) : d((uint32_t)by), mul(0), shift(0) {
    if (by <= 1) return;
    int l = 0;
    while ((int64_t(1) << l) < by) ++l;
    mul = (uint32_t)(((uint64_t(1) << (31 + l)) + d - 1) / d);
    shift = (uint32_t)(l - 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return mul ? __umulhi(n, mul) >> shift : n; }
#endif
};

// new rows of a cache in 8 bits (msm_qpages.cu)
struct QPagesWrite {
  PagesMeta m;
  int n_kv_heads, n_tokens, block_rows, page_blocks;
  int group;  // tokens that one unit of threads looks at
  Divisor by_page, by_block;  // page_rows, block_rows
  uint8_t *pool_k, *pool_v;
  float *k_scales, *v_scales;
  const uint16_t *k, *v;
  int64_t k_token, k_head, v_token, v_head;  // strides in elements
  const int32_t* starts;
};
cudaError_t launch_qpages_write(const QPagesWrite& p, int dtype, int head_dim, cudaStream_t s);

// attention of one new token per sequence (msm_paged_attn.cu)
struct PagedAttn {
  const int32_t *table, *lens;
  int32_t* status;
  int n_seqs, max_pages, n_pages, page_rows, n_kv_heads, group, window;
  int sinks;   // rows at the front that stay visible (0 without a window)
  int finish, solo_tiles;  // what an item costs beside its tiles, in tiles (1: one of at most solo_tiles tiles)
  const uint16_t* q;
  const void *k, *v;  // the layer's pools
  // a cache in 8 bits (else null): fp32 [n_pages][n_kv_heads][page_blocks], a scale for block_rows rows each
  const float *k_scales, *v_scales;
  int block_rows, page_blocks;
  Divisor by_page, by_block;  // page_rows, block_rows
  uint16_t* out;
  int64_t q_seq, q_head, out_seq, out_head;  // strides in elements
  float scale_log2;                          // softmax scale x log2(e)
  uint32_t* counters;                        // workspace: three per block, zero between calls,
  float* part;                               // and partial results, two per block
};
// what an item costs beside its tiles (PagedAttn::finish).  8 bits: its tiles are cheaper, its end is not (64 sequences of 1
// to 8,192 rows: 47 us with 1, 37 with 2, 34 with 4, 35 with 6, 37 with 9; that batch alone was looked at, 32 query heads on 8 of 128)
constexpr int kPagedFinish = 1, kQPagedFinish = 4;
// 8 bits: most tiles of an item that one warp does alone, which spares the block its barriers (512 sequences of 30 rows 50 -> 26
// us).  Up to three where there are many items, so that the warps' shares even out (512 of 1 to 200 rows: 66 us without, 63
// with one, 50 with three, 49 with five), one where there are few (64 of 1 to 8,192: 34 us without, 33 with one, 35 with
// three, 39 with five).  (These two batches were looked at, not head_dim 64, other groups or windows.)
constexpr int kQPagedSolo = 1, kQPagedSoloMany = 3, kQPagedMany = 8;  // (many: items per block)
constexpr int kPagedAttnPerSm = 2, kQPagedAttnPerSm = 2;  // blocks per SM (of 16 and of 8 bits)
size_t paged_attn_workspace(int blocks, int group, int head_dim);
cudaError_t launch_paged_attn(const PagedAttn& p, int dtype, int head_dim, int blocks, cudaStream_t s);

// what the page operations share: the status word
#ifdef __CUDACC__
__device__ __forceinline__ void latch(int32_t* status, int code, int call) {
  atomicCAS(status, 0, code | (call << 8));
}
// (only ever set by a call that the others are ordered behind, so all threads of a call see the same)
__device__ __forceinline__ bool stopped(const int32_t* status) { return (__ldcg(status) & kPagesStopped) != 0; }
#endif

// causal attention of packed prompts (msm_prompt.cu)
struct PromptAttn {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;  // strides in elements
  const int32_t *q_starts, *k_starts;
  int n_seqs, n_q, n_k, n_kv_heads, group, window;
  int sinks;         // keys at a sequence's front that stay visible behind the window (0 without a window; at most n_k)
  int out_32;        // every row of out starts on a 32-byte boundary
  float scale_log2;  // softmax scale x log2(e)
  int32_t* status;   // becomes MSM_ERR_DEVICE_TIMEOUT when a wait ran out (may be null)
  int drop;          // test hook: nothing is loaded
};
// most pieces of work that a call can have (its sequences' lengths are on the device); below 2^31 - 2^16
// for a launch
int64_t prompt_attn_works(int n_q, int n_seqs, int n_kv_heads, int group);
cudaError_t launch_prompt_attn(const PromptAttn& p, int dtype, int head_dim, int sms, cudaStream_t s);

cudaError_t launch_pages_resize(const PagesMeta& p, cudaStream_t s);
cudaError_t launch_pages_fork(const PagesMeta& p, cudaStream_t s);
cudaError_t launch_pages_compact(const PagesMeta& p, cudaStream_t s);
cudaError_t launch_pages_copy(const PagesCopy& p, bool compact, int sms, cudaStream_t s);
cudaError_t launch_pages_write(const PagesWrite& p, cudaStream_t s);

}  // namespace msm
