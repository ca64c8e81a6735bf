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
  uint4* k[kPagesLayers];
  uint4* v[kPagesLayers];
};

struct PagesWrite {
  PagesMeta m;
  int n_kv_heads, row_shift, n_tokens;  // 2^row_shift 16-byte vectors per row
  uint4 *pool_k, *pool_v;
  const uint4 *k, *v;
  int64_t k_token, k_head, v_token, v_head;  // strides in 16-byte vectors
  const int32_t* starts;
};

// attention of one new token per sequence (msm_paged_attn.cu)
struct PagedAttn {
  const int32_t *table, *lens;
  int32_t* status;
  int n_seqs, max_pages, n_pages, page_rows, n_kv_heads, group, window;
  const uint16_t *q, *k, *v;  // k, v: the layer's pools
  uint16_t* out;
  int64_t q_seq, q_head, out_seq, out_head;  // strides in elements
  float scale_log2;                          // softmax scale x log2(e)
  uint32_t* counters;                        // workspace: three per block, zero between calls,
  float* part;                               // and partial results, two per block
};
constexpr int kPagedAttnPerSm = 2;  // blocks per SM
size_t paged_attn_workspace(int blocks, int group, int head_dim);
cudaError_t launch_paged_attn(const PagedAttn& p, int dtype, int head_dim, int blocks, cudaStream_t s);

// causal attention of packed prompts (msm_prompt.cu)
struct PromptAttn {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;  // strides in elements
  const int32_t *q_starts, *k_starts;
  int n_seqs, n_q, n_k, n_kv_heads, group, window;
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
