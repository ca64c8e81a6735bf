// Host side of the paged caches, of the prompt attention and of sampling (declared in include/msm.h):
// every call checks its arguments, then enqueues its launches on the caller's stream; no
// call allocates, waits (msm_pages_sync aside) or keeps anything for the next one.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "msm.h"
#include "msm_paged.h"
#include "msm_sample.h"

using namespace msm;

namespace {

#define CKP(call)                                       \
  do {                                                  \
    cudaError_t e_ = (call);                            \
    if (e_ != cudaSuccess) return report_cuda(e_, #call); \
  } while (0)
#define REQUIRE(cond, st, msg) \
  do {                         \
    if (!(cond)) return report(st, msg); \
  } while (0)

// makes a device current for the length of a call
class DeviceGuard {
 public:
  cudaError_t enter(int device) {
    cudaError_t e = cudaGetDevice(&was_);
    if (e != cudaSuccess) return e;
    if (was_ == device) return cudaSuccess;
    e = cudaSetDevice(device);
    changed_ = e == cudaSuccess;
    return e;
  }
  ~DeviceGuard() {
    if (changed_) cudaSetDevice(was_);
  }

 private:
  int was_ = 0;
  bool changed_ = false;
};

// SM count of a device; MSM_ERR_UNSUPPORTED for anything but sm_103
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];
msm_status device_sms(int device, int* sms) {
  if (device < 0 || device >= kMaxDevices) return report(MSM_ERR_INVALID_ARG, "no such device");
  int n = g_sms[device].load(std::memory_order_relaxed);
  if (n == 0) {
    int ndev = 0, major = 0, minor = 0;
    CKP(cudaGetDeviceCount(&ndev));
    REQUIRE(device < ndev, MSM_ERR_INVALID_ARG, "no such device");
    CKP(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device));
    CKP(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device));
    REQUIRE(major == 10 && minor == 3, MSM_ERR_UNSUPPORTED, "libmsm is built for sm_103a (GB300) only");
    CKP(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device));
    g_sms[device].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return MSM_OK;
}

bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

bool is_16_bit(int dtype) { return dtype == MSM_BF16 || dtype == MSM_FP16; }

// what the caches of 16 and of 8 bits have in common
msm_status check_layout(const msm_pages* c) {
  REQUIRE(c->n_layers > 0 && c->n_pages > 0 && c->page_rows > 0 && c->n_kv_heads > 0 && c->head_dim > 0 &&
              c->n_seqs > 0 && c->max_pages > 0,
          MSM_ERR_INVALID_ARG, "pages: non-positive size");
  REQUIRE(c->head_dim == 64 || c->head_dim == 128, MSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  // (a token's elements are counted in 32 bits)
  REQUIRE(c->n_kv_heads < 65536, MSM_ERR_UNSUPPORTED, "pages: more than 65535 kv heads");
  REQUIRE((int64_t)c->n_seqs * c->max_pages < (int64_t(1) << 31), MSM_ERR_UNSUPPORTED, "pages: table too large");
  // (the kernels step past a sequence's end by up to a tile in 32 bits)
  REQUIRE((int64_t)c->max_pages * c->page_rows < (int64_t(1) << 31) - 4096, MSM_ERR_UNSUPPORTED,
          "pages: max_pages * page_rows too large");
  REQUIRE(c->n_pages < (1 << 30) && (double)c->n_pages * c->n_kv_heads * c->page_rows < 4294967296.0,
          MSM_ERR_UNSUPPORTED, "pages: pool too large");
  REQUIRE(c->k_pages && c->v_pages && c->table && c->lens && c->refs && c->status && c->scratch, MSM_ERR_INVALID_ARG,
          "pages: NULL pointer");
  for (int l = 0; l < c->n_layers; ++l) {
    REQUIRE(c->k_pages[l] && c->v_pages[l], MSM_ERR_INVALID_ARG, "pages: NULL pool pointer");
    REQUIRE(!misaligned(c->k_pages[l], 16) && !misaligned(c->v_pages[l], 16), MSM_ERR_INVALID_ARG,
            "pages: pools must be 16-byte aligned");
  }
  REQUIRE(!misaligned(c->table, 4) && !misaligned(c->lens, 4) && !misaligned(c->refs, 4) &&
              !misaligned(c->status, 4) && !misaligned(c->scratch, 4),
          MSM_ERR_INVALID_ARG, "pages: table, lens, refs, status and scratch must be 4-byte aligned");
  return MSM_OK;
}

msm_status check_pages(const msm_pages* c) {
  REQUIRE(c, MSM_ERR_INVALID_ARG, "pages is NULL");
  REQUIRE(is_16_bit(c->dtype), MSM_ERR_INVALID_ARG, "pages: dtype must be MSM_BF16 or MSM_FP16");
  return check_layout(c);
}

msm_status check_pages(const msm_qpages* c) {
  REQUIRE(c, MSM_ERR_INVALID_ARG, "qpages is NULL");
  REQUIRE(c->pages.dtype == MSM_E4M3, MSM_ERR_INVALID_ARG, "qpages: dtype must be MSM_E4M3");
  const msm_status st = check_layout(&c->pages);
  if (st != MSM_OK) return st;
  REQUIRE(c->block_rows > 0 && c->block_rows <= c->pages.page_rows, MSM_ERR_INVALID_ARG,
          "qpages: block_rows must be 1 to page_rows");
  REQUIRE(c->k_scales && c->v_scales, MSM_ERR_INVALID_ARG, "qpages: NULL pointer");
  for (int l = 0; l < c->pages.n_layers; ++l)
    REQUIRE(c->k_scales[l] && c->v_scales[l] && !misaligned(c->k_scales[l], 4) && !misaligned(c->v_scales[l], 4),
            MSM_ERR_INVALID_ARG, "qpages: scales are NULL or not 4-byte aligned");
  return MSM_OK;
}

const msm_pages* base(const msm_pages* c) { return c; }
const msm_pages* base(const msm_qpages* c) { return &c->pages; }
const msm_qpages* held8(const msm_pages*) { return nullptr; }
const msm_qpages* held8(const msm_qpages* c) { return c; }

int per_sm(const msm_pages*) { return kPagedAttnPerSm; }
int per_sm(const msm_qpages*) { return kQPagedAttnPerSm; }

int page_blocks(const msm_qpages* c) { return (c->pages.page_rows - 1) / c->block_rows + 1; }

PagesMeta meta(const msm_pages* c, const int32_t* arg) {
  PagesMeta m;
  m.table = c->table;
  m.lens = c->lens;
  m.refs = c->refs;
  m.status = c->status;
  m.scratch = c->scratch;
  m.arg = arg;
  m.n_pages = c->n_pages;
  m.page_rows = c->page_rows;
  m.n_seqs = c->n_seqs;
  m.max_pages = c->max_pages;
  return m;
}

msm_status copy_rows(const msm_pages* c, const msm_qpages* q, const PagesMeta& m, bool compact, int sms,
                     cudaStream_t s) {
  PagesCopy p;
  std::memset(&p, 0, sizeof(p));
  p.m = m;
  p.n_kv_heads = c->n_kv_heads;
  p.row_vecs = c->head_dim / (q ? 16 : 8);
  if (q) {
    p.block_rows = q->block_rows;
    p.page_blocks = page_blocks(q);
  }
  for (int l0 = 0; l0 < c->n_layers; l0 += kPagesLayers) {
    p.n_layers = std::min(kPagesLayers, c->n_layers - l0);
    p.renumber = l0 == 0;
    for (int l = 0; l < p.n_layers; ++l) {
      p.k[l] = static_cast<uint4*>(c->k_pages[l0 + l]);
      p.v[l] = static_cast<uint4*>(c->v_pages[l0 + l]);
      if (q) {
        p.k_scales[l] = q->k_scales[l0 + l];
        p.v_scales[l] = q->v_scales[l0 + l];
      }
    }
    CKP(launch_pages_copy(p, compact, sms, s));
  }
  return MSM_OK;
}

bool bad_stride(int64_t st, int64_t least) { return st < least || st % 8 != 0 || st >= (int64_t(1) << 31); }

msm_status check_group(int n_q_heads, int n_kv_heads) {
  REQUIRE(n_q_heads > 0 && n_q_heads % n_kv_heads == 0, MSM_ERR_INVALID_ARG, "n_q_heads must be a multiple of n_kv_heads");
  const int group = n_q_heads / n_kv_heads;
  REQUIRE(group == 1 || group == 2 || group == 4 || group == 8, MSM_ERR_UNSUPPORTED,
          "n_q_heads / n_kv_heads must be 1, 2, 4 or 8");
  return MSM_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

// ---- the calls on a cache, of 16 bits (Cache = msm_pages) or of 8 (msm_qpages)
template <class Cache>
msm_status resize(const Cache* c, const int32_t* new_lens, void* stream) {
  msm_status st = check_pages(c);
  if (st != MSM_OK) return st;
  REQUIRE(new_lens && !misaligned(new_lens, 4), MSM_ERR_INVALID_ARG, "new_lens is NULL or misaligned");
  int sms = 0;
  if ((st = device_sms(base(c)->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(base(c)->device));
  const PagesMeta m = meta(base(c), new_lens);
  CKP(launch_pages_resize(m, static_cast<cudaStream_t>(stream)));
  return copy_rows(base(c), held8(c), m, false, sms, static_cast<cudaStream_t>(stream));
}

template <class Cache>
msm_status fork(const Cache* c, const int32_t* parent, void* stream) {
  msm_status st = check_pages(c);
  if (st != MSM_OK) return st;
  REQUIRE(parent && !misaligned(parent, 4), MSM_ERR_INVALID_ARG, "parent is NULL or misaligned");
  int sms = 0;
  if ((st = device_sms(base(c)->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(base(c)->device));
  CKP(launch_pages_fork(meta(base(c), parent), static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

template <class Cache>
msm_status compact(const Cache* c, void* stream) {
  msm_status st = check_pages(c);
  if (st != MSM_OK) return st;
  int sms = 0;
  if ((st = device_sms(base(c)->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(base(c)->device));
  const PagesMeta m = meta(base(c), nullptr);
  CKP(launch_pages_compact(m, static_cast<cudaStream_t>(stream)));
  return copy_rows(base(c), held8(c), m, true, sms, static_cast<cudaStream_t>(stream));
}

// the rows and strides of msm_pages_write and msm_qpages_write (n_tokens > 0)
msm_status check_rows(const void* k, const void* v, int64_t k_token_stride, int64_t k_head_stride,
                      int64_t v_token_stride, int64_t v_head_stride) {
  REQUIRE(k && v && !misaligned(k, 16) && !misaligned(v, 16), MSM_ERR_INVALID_ARG, "k or v is NULL or misaligned");
  REQUIRE(!bad_stride(k_token_stride, 0) && !bad_stride(k_head_stride, 0) && !bad_stride(v_token_stride, 0) &&
              !bad_stride(v_head_stride, 0),
          MSM_ERR_INVALID_ARG, "strides must be multiples of 8, not negative and below 2^31");
  return MSM_OK;
}

template <class Cache>
size_t attention_workspace(const Cache* c, int n_q_heads) {
  if (check_pages(c) != MSM_OK || check_group(n_q_heads, base(c)->n_kv_heads) != MSM_OK) return 0;
  int sms = 0;
  if (device_sms(base(c)->device, &sms) != MSM_OK) return 0;
  return paged_attn_workspace(sms * per_sm(c), n_q_heads / base(c)->n_kv_heads, base(c)->head_dim);
}

template <class Cache>
msm_status attention(const Cache* cache, int layer, int dtype, const void* q, int64_t q_seq_stride,
                     int64_t q_head_stride, int n_q_heads, float scale, int window, int sinks, void* out,
                     int64_t out_seq_stride, int64_t out_head_stride, void* workspace, size_t workspace_bytes,
                     void* stream) {
  msm_status st = check_pages(cache);
  if (st != MSM_OK) return st;
  const msm_pages* const c = base(cache);
  REQUIRE(layer >= 0 && layer < c->n_layers, MSM_ERR_INVALID_ARG, "layer out of range");
  REQUIRE(is_16_bit(dtype), MSM_ERR_INVALID_ARG, "dtype must be MSM_BF16 or MSM_FP16");
  if ((st = check_group(n_q_heads, c->n_kv_heads)) != MSM_OK) return st;
  REQUIRE(q && out && !misaligned(q, 16) && !misaligned(out, 16), MSM_ERR_INVALID_ARG, "q or out is NULL or misaligned");
  REQUIRE(!bad_stride(q_seq_stride, 0) && !bad_stride(q_head_stride, 0), MSM_ERR_INVALID_ARG,
          "strides must be multiples of 8, not negative and below 2^31");
  REQUIRE(!bad_stride(out_seq_stride, c->head_dim) && !bad_stride(out_head_stride, c->head_dim), MSM_ERR_INVALID_ARG,
          "strides of out must be multiples of 8, at least head_dim and below 2^31");
  REQUIRE(std::isfinite(scale * kLog2e), MSM_ERR_INVALID_ARG, "scale must be finite");
  REQUIRE(window >= 0, MSM_ERR_INVALID_ARG, "window is negative");
  REQUIRE(sinks >= 0, MSM_ERR_INVALID_ARG, "sinks is negative");
  REQUIRE(workspace && !misaligned(workspace, 16), MSM_ERR_INVALID_ARG, "workspace is NULL or misaligned");
  int sms = 0;
  if ((st = device_sms(c->device, &sms)) != MSM_OK) return st;
  const int blocks = sms * per_sm(cache), group = n_q_heads / c->n_kv_heads;
  REQUIRE(workspace_bytes >= paged_attn_workspace(blocks, group, c->head_dim), MSM_ERR_INVALID_ARG,
          "workspace is smaller than msm_paged_attention_workspace");
  DeviceGuard dev;
  CKP(dev.enter(c->device));
  PagedAttn p;
  p.table = c->table;
  p.lens = c->lens;
  p.status = c->status;
  p.n_seqs = c->n_seqs;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.page_rows = c->page_rows;
  p.n_kv_heads = c->n_kv_heads;
  p.group = group;
  p.window = window;
  p.sinks = window > 0 ? sinks : 0;
  p.finish = held8(cache) ? kQPagedFinish : kPagedFinish;
  p.solo_tiles = !held8(cache) ? 0 : (int64_t)c->n_seqs * c->n_kv_heads < (int64_t)kQPagedMany * blocks ? kQPagedSolo : kQPagedSoloMany;
  p.q = static_cast<const uint16_t*>(q);
  p.k = c->k_pages[layer];
  p.v = c->v_pages[layer];
  p.k_scales = p.v_scales = nullptr;
  p.block_rows = p.page_blocks = 0;
  p.by_page = Divisor(c->page_rows);
  if (const msm_qpages* const h = held8(cache)) {
    p.k_scales = h->k_scales[layer];
    p.v_scales = h->v_scales[layer];
    p.block_rows = h->block_rows;
    p.page_blocks = page_blocks(h);
    p.by_block = Divisor(h->block_rows);
  }
  p.out = static_cast<uint16_t*>(out);
  p.q_seq = q_seq_stride;
  p.q_head = q_head_stride;
  p.out_seq = out_seq_stride;
  p.out_head = out_head_stride;
  p.scale_log2 = scale * kLog2e;
  p.part = static_cast<float*>(workspace);
  p.counters = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) +
                                           paged_attn_workspace(blocks, group, c->head_dim)) - 3 * blocks;
  CKP(launch_paged_attn(p, dtype, c->head_dim, blocks, static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

template <class Cache>
msm_status sync(const Cache* cache, void* stream) {
  msm_status st = check_pages(cache);
  if (st != MSM_OK) return st;
  const msm_pages* const c = base(cache);
  int sms = 0;
  if ((st = device_sms(c->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(c->device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  CKP(cudaMemcpyAsync(&word, c->status, sizeof(word), cudaMemcpyDeviceToHost, s));
  CKP(cudaStreamSynchronize(s));
  if (word == 0) return MSM_OK;
  CKP(cudaMemsetAsync(c->status, 0, sizeof(word), s));
  CKP(cudaStreamSynchronize(s));
  const int code = word & 0xFF, call = word >> 8 & 0xFF;
  const char* const pages = held8(cache) ? "msm_qpages" : "msm_pages";
  char buf[128];
  const char* const why = code == MSM_ERR_OOM ? "no free page left" : "lengths, parents or table entries out of range";
  if (call == kCallAttention)
    std::snprintf(buf, sizeof(buf), "%s: %s", held8(cache) ? "msm_qpages_attention" : "msm_paged_attention", why);
  else
    std::snprintf(buf, sizeof(buf), "%s_%s: %s", pages,
                  call == kCallResize ? "resize"
                  : call == kCallFork ? "fork"
                  : call == kCallWrite ? "write"
                                       : "unknown call",
                  why);
  return report(code == MSM_ERR_OOM ? MSM_ERR_OOM : code == MSM_ERR_INVALID_ARG ? MSM_ERR_INVALID_ARG : MSM_ERR_CUDA,
                buf);
}
}  // namespace

extern "C" {

size_t msm_pages_scratch_ints(int n_pages, int n_seqs) {
  return n_pages > 0 && n_seqs > 0 ? pages_scratch_ints(n_pages, n_seqs) : 0;
}

msm_status msm_pages_resize(const msm_pages* c, const int32_t* new_lens, void* stream) { return resize(c, new_lens, stream); }
msm_status msm_pages_fork(const msm_pages* c, const int32_t* parent, void* stream) { return fork(c, parent, stream); }
msm_status msm_pages_compact(const msm_pages* c, void* stream) { return compact(c, stream); }
msm_status msm_pages_sync(const msm_pages* c, void* stream) { return sync(c, stream); }
msm_status msm_qpages_resize(const msm_qpages* c, const int32_t* new_lens, void* stream) { return resize(c, new_lens, stream); }
msm_status msm_qpages_fork(const msm_qpages* c, const int32_t* parent, void* stream) { return fork(c, parent, stream); }
msm_status msm_qpages_compact(const msm_qpages* c, void* stream) { return compact(c, stream); }
msm_status msm_qpages_sync(const msm_qpages* c, void* stream) { return sync(c, stream); }

msm_status msm_pages_write(const msm_pages* c, int layer, const void* k, const void* v, int64_t k_token_stride,
                           int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t* starts, int n_tokens, void* stream) {
  msm_status st = check_pages(c);
  if (st != MSM_OK) return st;
  REQUIRE(layer >= 0 && layer < c->n_layers, MSM_ERR_INVALID_ARG, "layer out of range");
  REQUIRE(n_tokens >= 0, MSM_ERR_INVALID_ARG, "n_tokens is negative");
  REQUIRE(starts && !misaligned(starts, 4), MSM_ERR_INVALID_ARG, "starts is NULL or misaligned");
  if (n_tokens == 0) return MSM_OK;
  if ((st = check_rows(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride)) != MSM_OK) return st;
  int sms = 0;
  if ((st = device_sms(c->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(c->device));
  PagesWrite p;
  p.m = meta(c, nullptr);
  p.n_kv_heads = c->n_kv_heads;
  p.row_shift = c->head_dim == 64 ? 3 : 4;
  p.n_tokens = n_tokens;
  p.pool_k = static_cast<uint4*>(c->k_pages[layer]);
  p.pool_v = static_cast<uint4*>(c->v_pages[layer]);
  p.k = static_cast<const uint4*>(k);
  p.v = static_cast<const uint4*>(v);
  p.k_token = k_token_stride / 8;
  p.k_head = k_head_stride / 8;
  p.v_token = v_token_stride / 8;
  p.v_head = v_head_stride / 8;
  p.starts = starts;
  CKP(launch_pages_write(p, static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

msm_status msm_qpages_write(const msm_qpages* c, int layer, int dtype, const void* k, const void* v,
                            int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                            int64_t v_head_stride, const int32_t* starts, int n_tokens, void* stream) {
  msm_status st = check_pages(c);
  if (st != MSM_OK) return st;
  REQUIRE(layer >= 0 && layer < c->pages.n_layers, MSM_ERR_INVALID_ARG, "layer out of range");
  REQUIRE(is_16_bit(dtype), MSM_ERR_INVALID_ARG, "dtype must be MSM_BF16 or MSM_FP16");
  REQUIRE(n_tokens >= 0, MSM_ERR_INVALID_ARG, "n_tokens is negative");
  REQUIRE(starts && !misaligned(starts, 4), MSM_ERR_INVALID_ARG, "starts is NULL or misaligned");
  if (n_tokens == 0) return MSM_OK;
  if ((st = check_rows(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride)) != MSM_OK) return st;
  int sms = 0;
  if ((st = device_sms(c->pages.device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(c->pages.device));
  QPagesWrite p;
  p.m = meta(&c->pages, nullptr);
  p.n_kv_heads = c->pages.n_kv_heads;
  p.n_tokens = n_tokens;
  p.block_rows = c->block_rows;
  p.page_blocks = page_blocks(c);
  // a sequence's tokens in groups of a block's; a step's few tokens one by one
  p.group = std::max(1, std::min(c->block_rows, n_tokens / c->pages.n_seqs));
  p.by_page = Divisor(c->pages.page_rows);
  p.by_block = Divisor(c->block_rows);
  p.pool_k = static_cast<uint8_t*>(c->pages.k_pages[layer]);
  p.pool_v = static_cast<uint8_t*>(c->pages.v_pages[layer]);
  p.k_scales = c->k_scales[layer];
  p.v_scales = c->v_scales[layer];
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  p.starts = starts;
  CKP(launch_qpages_write(p, dtype, c->pages.head_dim, static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

size_t msm_paged_attention_workspace(const msm_pages* c, int n_q_heads) { return attention_workspace(c, n_q_heads); }
size_t msm_qpages_attention_workspace(const msm_qpages* c, int n_q_heads) { return attention_workspace(c, n_q_heads); }

msm_status msm_paged_attention_sinks(const msm_pages* c, int layer, const void* q, int64_t q_seq_stride,
                                     int64_t q_head_stride, int n_q_heads, float scale, int window, int sinks,
                                     void* out, int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return attention(c, layer, c ? c->dtype : MSM_BF16, q, q_seq_stride, q_head_stride, n_q_heads, scale, window, sinks,
                   out, out_seq_stride, out_head_stride, workspace, workspace_bytes, stream);
}

msm_status msm_paged_attention(const msm_pages* c, int layer, const void* q, int64_t q_seq_stride,
                               int64_t q_head_stride, int n_q_heads, float scale, int window, void* out,
                               int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return msm_paged_attention_sinks(c, layer, q, q_seq_stride, q_head_stride, n_q_heads, scale, window, 0, out,
                                   out_seq_stride, out_head_stride, workspace, workspace_bytes, stream);
}

msm_status msm_qpages_attention(const msm_qpages* c, int layer, int dtype, const void* q, int64_t q_seq_stride,
                                int64_t q_head_stride, int n_q_heads, float scale, int window, int sinks, void* out,
                                int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return attention(c, layer, dtype, q, q_seq_stride, q_head_stride, n_q_heads, scale, window, sinks, out,
                   out_seq_stride, out_head_stride, workspace, workspace_bytes, stream);
}

msm_status msm_prompt_attention(const msm_prompt* a, void* stream) { return msm_prompt_attention_sinks(a, 0, stream); }

msm_status msm_prompt_attention_sinks(const msm_prompt* a, int sinks, void* stream) {
  REQUIRE(a, MSM_ERR_INVALID_ARG, "prompt is NULL");
  REQUIRE(a->dtype == MSM_BF16 || a->dtype == MSM_FP16, MSM_ERR_INVALID_ARG, "prompt: dtype must be MSM_BF16 or MSM_FP16");
  REQUIRE(a->n_seqs > 0 && a->n_q >= 0 && a->n_k >= 0 && a->n_q_heads > 0 && a->n_kv_heads > 0 && a->head_dim > 0,
          MSM_ERR_INVALID_ARG, "prompt: a size is out of range");
  REQUIRE(a->head_dim == 64 || a->head_dim == 128, MSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  msm_status st = check_group(a->n_q_heads, a->n_kv_heads);
  if (st != MSM_OK) return st;
  REQUIRE(a->n_q < (1 << 27) && a->n_k < (1 << 27) && a->n_kv_heads < 65536, MSM_ERR_UNSUPPORTED,
          "prompt: more than 2^27 tokens or 65535 kv heads");
  REQUIRE(prompt_attn_works(a->n_q, a->n_seqs, a->n_kv_heads, a->n_q_heads / a->n_kv_heads) < 0x7FFF0000,
          MSM_ERR_UNSUPPORTED, "prompt: too many sequences times kv heads");
  REQUIRE(a->window >= 0, MSM_ERR_INVALID_ARG, "window is negative");
  REQUIRE(sinks >= 0, MSM_ERR_INVALID_ARG, "sinks is negative");
  REQUIRE(std::isfinite(a->scale * kLog2e), MSM_ERR_INVALID_ARG, "scale must be finite");
  if (a->n_q == 0) return MSM_OK;
  REQUIRE(a->q && a->out && a->q_starts && a->k_starts && (a->n_k == 0 || (a->k && a->v)), MSM_ERR_INVALID_ARG,
          "prompt: NULL pointer");
  REQUIRE(!misaligned(a->q, 16) && !misaligned(a->k, 16) && !misaligned(a->v, 16) && !misaligned(a->out, 16) &&
              !misaligned(a->q_starts, 4) && !misaligned(a->k_starts, 4) && !misaligned(a->status, 4),
          MSM_ERR_INVALID_ARG, "prompt: q, k, v and out must be 16-byte, the starts and status 4-byte aligned");
  REQUIRE((a->flags & ~MSM_FLAG_TEST_DROP_HANDOFF) == 0, MSM_ERR_INVALID_ARG, "prompt: unknown flags");
  const int64_t strides[] = {a->q_token_stride, a->q_head_stride, a->k_token_stride, a->k_head_stride,
                             a->v_token_stride, a->v_head_stride, a->out_token_stride, a->out_head_stride};
  for (int64_t s : strides)
    REQUIRE(!bad_stride(s, a->head_dim), MSM_ERR_INVALID_ARG,
            "prompt: strides must be multiples of 8, at least head_dim and below 2^31");
  int sms = 0;
  if ((st = device_sms(a->device, &sms)) != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(a->device));
  PromptAttn p;
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.q_token = a->q_token_stride;
  p.q_head = a->q_head_stride;
  p.k_token = a->k_token_stride;
  p.k_head = a->k_head_stride;
  p.v_token = a->v_token_stride;
  p.v_head = a->v_head_stride;
  p.out_token = a->out_token_stride;
  p.out_head = a->out_head_stride;
  p.out_32 = !misaligned(a->out, 32) && a->out_token_stride % 16 == 0 && a->out_head_stride % 16 == 0;
  p.q_starts = a->q_starts;
  p.k_starts = a->k_starts;
  p.n_seqs = a->n_seqs;
  p.n_q = a->n_q;
  p.n_k = a->n_k;
  p.n_kv_heads = a->n_kv_heads;
  p.group = a->n_q_heads / a->n_kv_heads;
  // (a window of all keys hides none, nor does one behind as many sinks; the kernel's differences of positions and a smaller one stay
  // far inside 32 bits, also for queries in front of the first key)
  p.window = a->window < a->n_k && sinks < a->n_k ? a->window : 0;
  p.sinks = p.window > 0 ? sinks : 0;
  p.scale_log2 = a->scale * kLog2e;
  p.status = a->status;
  p.drop = (a->flags & MSM_FLAG_TEST_DROP_HANDOFF) != 0;
  CKP(launch_prompt_attn(p, a->dtype, a->head_dim, sms, static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

msm_status msm_sample(const msm_sampling* a, void* stream) {
  REQUIRE(a, MSM_ERR_INVALID_ARG, "sampling is NULL");
  REQUIRE(is_16_bit(a->dtype) || a->dtype == MSM_FP32, MSM_ERR_INVALID_ARG,
          "sampling: dtype must be MSM_FP32, MSM_BF16 or MSM_FP16");
  REQUIRE(a->n_rows >= 0 && a->vocab > 0, MSM_ERR_INVALID_ARG, "sampling: a size is out of range");
  REQUIRE(a->vocab <= kSampleVocab && a->n_rows < (1 << 24), MSM_ERR_UNSUPPORTED,
          "sampling: more than 2^20 logits in a row, or 2^24 rows");
  REQUIRE(a->row_stride >= 0, MSM_ERR_INVALID_ARG, "sampling: row_stride is negative");
  if (a->n_rows == 0) return MSM_OK;
  REQUIRE(a->logits && a->random && a->tokens, MSM_ERR_INVALID_ARG, "sampling: NULL pointer");
  REQUIRE(!misaligned(a->logits, a->dtype == MSM_FP32 ? 4 : 2) && !misaligned(a->temperature, 4) &&
              !misaligned(a->top_k, 4) && !misaligned(a->top_p, 4) && !misaligned(a->min_p, 4) &&
              !misaligned(a->random, 4) && !misaligned(a->tokens, 4) && !misaligned(a->probs, 4) &&
              !misaligned(a->kept, 4),
          MSM_ERR_INVALID_ARG, "sampling: a pointer is not aligned to its type");
  int sms = 0;
  msm_status st = device_sms(a->device, &sms);
  if (st != MSM_OK) return st;
  DeviceGuard dev;
  CKP(dev.enter(a->device));
  SampleArgs p;
  p.logits = a->logits;
  p.stride = a->row_stride;
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.random = a->random;
  p.tokens = a->tokens;
  p.kept = a->kept;
  p.probs = a->probs;
  p.n_rows = a->n_rows;
  p.vocab = a->vocab;
  p.slice = p.room = 0;
  CKP(launch_sample(p, a->dtype, sms, static_cast<cudaStream_t>(stream)));
  return MSM_OK;
}

}  // extern "C"
