/*
 * msm.h — C ABI of libmsm: one speculative-decoding verify step of a batch-1
 * mixture-of-experts decoder on one GB300 GPU, one persistent kernel launch per
 * decoder layer.
 *
 * The method (LMSYS/SGLang megakernel for "Muse Spark Open", as reported by the
 * alphasignal.ai article "LMSYS Doubles Muse Spark Open Speed to 1,109 Tokens per
 * Second" and the orcarouter.ai article "Muse Spark Open: 1,109 tokens/s is a
 * kernel-level change"):
 *   - the target model verifies a 16-token tree proposed by a draft model in one
 *     pass (alphasignal.ai, § "Draft and verify share one graph"; orcarouter.ai,
 *     § on the draft model: the candidates form a tree, not a linear chain);
 *   - each launch covers one decoder layer's attention through the next layer's
 *     QKV projection and KV-cache write (alphasignal.ai, § "Launch boundaries
 *     leave hardware idle"; orcarouter.ai, § "where the kernel boundary sits");
 *   - the layer: tree-masked attention over the KV history (46 sliding-window
 *     layers over the last 2,048 tokens, 16 global), output projection, pooler,
 *     router top-8 of 256, two NVFP4 expert GEMMs, unpooler and combine
 *     (orcarouter.ai, § "where the kernel boundary sits").
 *
 * Conventions
 *   - Every call is host-synchronous in its validation and asynchronous on the
 *     stream it is given for GPU work.  Host-detectable errors (null pointers,
 *     invalid parent array, positions out of range, unsupported widths) return
 *     at once without enqueuing anything.
 *   - Device pointers are passed as plain pointers; `stream` is a cudaStream_t
 *     passed as void* (NULL = legacy default stream).
 *   - The caller owns every buffer it passes: weights (only read during
 *     msm_model_create, which copies them into a packed, model-owned layout —
 *     they may be freed once it returns), KV caches, hidden states, logits.
 *   - The model owns its packed weights, exchange buffers, routing records,
 *     timing buffer and device status word.
 *   - Bounded device waits: every in-kernel wait gives up after
 *     msm_config.timeout_us, records MSM_ERR_DEVICE_TIMEOUT in the model's status
 *     word and lets the launch finish; msm_sync() reports it and re-arms the
 *     model.  Nothing traps.
 *   - A model is not thread-safe; one model may be used by one host thread at a
 *     time.  Two steps of one model must not overlap on the GPU.
 *   - Co-residency: the blocks of a layer launch (one per SM, grid_blocks of them)
 *     wait on each other, so all of them must be resident at once.  The model checks
 *     at creation that the grid fits the device (one 384-thread block with ~227 KB
 *     of shared memory per SM); while steps run, nothing else may occupy the SMs
 *     (another kernel, another model's step, MPS or MIG clients).  If blocks cannot
 *     be co-resident, the bounded waits run out and the step reports
 *     MSM_ERR_DEVICE_TIMEOUT instead of hanging.
 *
 * Layouts (row-major; "bf16" is the 16-bit brain-float bit pattern)
 *   hidden state      bf16 [16][d_model]        (tree token i in row i)
 *   parent            int32 [16] host array: parent[0] == -1, 0 <= parent[i] < i
 *   KV cache (layer)  bf16 [n_kv_heads][max_ctx][head_dim]; rows [0, pos0) hold
 *                     the history (K already rotated); the step writes the K/V of
 *                     tree token i to row pos0 + i
 *   logits            fp32 [16][vocab]
 *   w_qkv             bf16 [(n_q_heads + 2 n_kv_heads) head_dim][d_model]
 *                     (rows: q heads, then k heads, then v heads)
 *   w_o               bf16 [d_model][n_q_heads head_dim]
 *   w_pool            bf16 [pool_dim][d_model]
 *   w_router          bf16 [n_experts][pool_dim];  b_router fp32 [n_experts]
 *   w_unpool          bf16 [d_model][pool_dim]
 *   norm_attn/norm_moe/norm_final  bf16 [d_model] RMSNorm gains
 *   w1 (NVFP4)        codes uint8 [n_experts][2 ffn_dim][pool_dim/2] (two E2M1
 *                     codes per byte, low nibble = even column), block scales
 *                     unsigned E4M3 (UE4M3: bit 7 must be 0 and is ignored)
 *                     [n_experts][2 ffn_dim][pool_dim/16], tensor scale fp32
 *                     [n_experts]; rows [0, ffn_dim) = SwiGLU gate, the rest = up
 *   w2 (NVFP4)        codes [n_experts][pool_dim][ffn_dim/2], scales
 *                     [n_experts][pool_dim][ffn_dim/16], tensor scale [n_experts]
 *   w_lm              bf16 [vocab][d_model]
 */
#ifndef MSM_H
#define MSM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSM_TREE_TOKENS 16

typedef enum {
  MSM_OK = 0,
  MSM_ERR_INVALID_ARG = 1,    /* bad pointer, parent array, position or config */
  MSM_ERR_CUDA = 2,           /* a CUDA runtime call failed (see msm_last_error) */
  MSM_ERR_OOM = 3,            /* device allocation failed */
  MSM_ERR_DEVICE_TIMEOUT = 4, /* a bounded in-kernel wait expired */
  MSM_ERR_UNSUPPORTED = 5     /* widths / features this library does not implement */
} msm_status;

/* msm_config.flags */
#define MSM_FLAG_SELF_TIMING 0x1u      /* %globaltimer stamps per block and phase (the
                                          orcarouter.ai article, § "where the 5.9 ms
                                          still goes": the kernel times itself) */
#define MSM_FLAG_EXPERT_PREFETCH 0x2u  /* L2 prefetch of the previous step's most-used
                                          experts (alphasignal.ai, § "Four mechanisms
                                          keep work moving") */
#define MSM_FLAG_KV_PREFETCH 0x4u      /* L2 prefetch of the next layer's KV history at
                                          combine time (orcarouter.ai, § "where the
                                          5.9 ms still goes") */
#define MSM_FLAG_PDL 0x8u              /* chain layer launches with programmatic
                                          dependent launch */
#define MSM_FLAG_DRAFT 0x20u           /* the model is the draft model of the decode
                                          step (alphasignal.ai, § "Draft and verify share
                                          one graph"): each layer's MoE half is a dense
                                          SwiGLU FFN (w_gate, w_up, w_down; norm_moe is
                                          its RMSNorm gain), every layer attends to its
                                          whole KV history and to all 16 slots of the
                                          block (no tree mask, no window); pool_dim,
                                          n_experts and top_k are 0 and the expert,
                                          pooler, router and unpooler weights NULL;
                                          vocab > 0.  Run with msm_draft_step. */
#define MSM_FLAG_TEST_DROP_HANDOFF 0x10000u /* test hook: one block never signals that
                                          its share of h1 is stored, so the pooler's
                                          consumers time out */

typedef struct {
  int d_model, n_q_heads, n_kv_heads, head_dim;
  int pool_dim, ffn_dim, n_experts, top_k;
  int n_layers;
  int vocab;        /* 0: no LM head; the step then returns the final hidden state */
  int window;       /* sliding window (keys r with tpos - r < window) of non-global layers */
  int max_ctx;      /* KV rows per layer and head */
  const uint8_t* layer_is_global; /* host [n_layers]: 1 = global attention */
  float rms_eps, rope_theta;
  uint32_t flags;   /* MSM_FLAG_* */
  int grid_blocks;  /* persistent blocks per launch; 0 = one per SM */
  int attn_splits;  /* KV splits per kv head; 0 = automatic */
  int prefetch_experts; /* experts prefetched by MSM_FLAG_EXPERT_PREFETCH; 0 = 14 */
  uint32_t timeout_us;  /* bounded-wait limit; 0 = 200000 */
  int l2_runahead_kb;   /* L2 prefetch distance of each block's dense-weight / KV
                           stream (expert tiles are not prefetched), KiB; 0 = off
                           (alphasignal.ai, § "Four mechanisms keep work moving":
                           weights for the next operation are fetched while the
                           current one runs, partly staged in L2).  Measured slower
                           than off on the 62-layer workload (32 KiB: +7 %), hence off. */
} msm_config;

/* Device pointers, one per layer (host arrays of n_layers entries). */
typedef struct {
  const void* const* w_qkv;
  const void* const* w_o;
  const void* const* w_pool;
  const void* const* w_router;
  const float* const* b_router;
  const void* const* w_unpool;
  const void* const* norm_attn;
  const void* const* norm_moe;
  const uint8_t* const* w1_codes;
  const uint8_t* const* w1_scales;
  const float* const* w1_tensor_scale;
  const uint8_t* const* w2_codes;
  const uint8_t* const* w2_scales;
  const float* const* w2_tensor_scale;
  const void* norm_final; /* required when vocab > 0 */
  const void* w_lm;       /* required when vocab > 0 */
  /* MSM_FLAG_DRAFT models only (NULL otherwise): bf16 [ffn_dim][d_model] gate and up
     projections and bf16 [d_model][ffn_dim] down projection of each layer's FFN */
  const void* const* w_gate;
  const void* const* w_up;
  const void* const* w_down;
} msm_weights;

typedef struct msm_model msm_model;

/* Statistics of the model and of its last step (host struct). */
typedef struct {
  int grid_blocks, threads_per_block, smem_bytes, attn_splits;
  int launches_per_step;         /* kernel launches one msm_verify_step enqueues */
  int cooperative;               /* 1 if launches are cooperative (co-residency guaranteed) */
  uint64_t packed_weight_bytes;  /* model-owned packed weights */
  uint64_t exchange_bytes;       /* model-owned exchange buffers */
  int tma_act_staging;           /* 1 if dense activations are staged by tensor copies
                                    (msm_verify_step / _dev), 0 if by plain loads */
  uint64_t launches_run;         /* layer-kernel launches enqueued so far by every verify
                                    entry point (a graph capture records, not runs) */
  uint64_t noalloc_scratch_bytes;  /* static scratch one msm_verify_step_noalloc call needs */
} msm_stats;

/*
 * Create a model on `device`: validate the config, pack the caller's weights
 * into the model's layout (GPU kernels on an internal stream, completed before
 * return) and allocate the exchange buffers.
 * Errors: MSM_ERR_INVALID_ARG (null pointer, bad config), MSM_ERR_UNSUPPORTED
 * (widths outside what the kernels implement: d_model and n_q_heads*head_dim
 * multiples of 64, pool_dim and ffn_dim multiples of 256 with pool_dim <= 2048
 * and ffn_dim <= 1024, head_dim 64 or 128, n_q_heads/n_kv_heads in {1,2,4,8},
 * top_k <= 8, n_experts <= 256 and a multiple of 16, vocab a multiple of 16; a
 * grid larger than the device keeps resident), MSM_ERR_OOM, MSM_ERR_CUDA.  On
 * error *out is NULL.
 */
msm_status msm_model_create(const msm_config* config, const msm_weights* weights, int device,
                            msm_model** out);

/* Free every model-owned buffer.  Waits for the model's work to finish.  NULL is ignored. */
void msm_model_destroy(msm_model* model);

/*
 * One verify step: for every layer in order, tree attention over the cache rows
 * [0, pos0) and the tree's own rows, then the MoE block; writes the K/V rows of
 * the 16 tree tokens to rows pos0..pos0+15 of every layer's cache, and the
 * logits of all 16 tree tokens (vocab > 0) and/or the final hidden state.
 *   hidden_in   device bf16 [16][d_model] (read)
 *   parent      host int32 [16]; parent[0] == -1, 0 <= parent[i] < i
 *   pos0        first tree row; 0 <= pos0 and pos0 + 16 <= max_ctx
 *   k_cache, v_cache  host arrays of n_layers device pointers (see layout)
 *   logits_out  device fp32 [16][vocab] or NULL (must be non-NULL if vocab > 0)
 *   hidden_out  device bf16 [16][d_model] or NULL (must be non-NULL if vocab == 0)
 * Enqueues n_layers launches on `stream`.  Device-side failures are reported
 * by the next msm_sync().
 */
msm_status msm_verify_step(msm_model* model, const void* hidden_in, const int32_t* parent,
                           int32_t pos0, void* const* k_cache, void* const* v_cache,
                           float* logits_out, void* hidden_out, void* stream);

/*
 * The same step with hidden_in / logits_out / hidden_out in HOST memory: copies
 * the input to the device, runs the step, copies the results back and waits
 * for the stream.  Returns the step's device status as msm_sync() would.
 * Host buffers may be pageable; pinned buffers make the copies asynchronous.
 */
msm_status msm_verify_step_host(msm_model* model, const void* hidden_in_host,
                                const int32_t* parent, int32_t pos0, void* const* k_cache,
                                void* const* v_cache, float* logits_host, void* hidden_out_host,
                                void* stream);

/*
 * msm_verify_step_noalloc: the verify step of msm_verify_step (same arguments,
 * same results, bit for bit) with its per-step scratch taken from a fixed
 * static device array instead of the model's own buffers.  The pages describe
 * no such entry point; it has no counterpart there.
 *
 * Who needs it: callers that must not allocate device memory at the time they
 * run a step -- for instance code under a strict device-memory budget, or code
 * that pre-plans all of its memory and forbids allocation on the decode path.
 * On success this call allocates nothing: no cudaMalloc / cudaFree, no
 * allocating library call.  (msm_verify_step allocates nothing per step either,
 * but it uses exchange buffers that msm_model_create allocated for the model;
 * this entry point uses the static array instead.)
 *
 * Scratch: MSM_NOALLOC_SCRATCH_BYTES (10 MiB) of __device__ memory per device,
 * shared by every model on that device.  A step needs
 *   2 * (exchange buffers + 256 bytes of phase counters) + attention/expert
 *   partials + 2 * (16 n_q_heads head_dim * 2) + 2 * (16 d_model * 2) bytes
 * (each part rounded up to 256 bytes), about 8.4 MiB at d_model 4096, 32/8
 * heads of 128, pool_dim 2048, ffn_dim 1024, top-8 on 152 SMs; the exact
 * figure of a model is msm_stats.noalloc_scratch_bytes.  A model whose step
 * needs more is rejected with MSM_ERR_UNSUPPORTED and a message giving both
 * sizes; nothing is launched.
 * The exchange part must hold its empty sentinels when a step starts; every
 * call arms it on `stream` before its first layer launch, so no state carries
 * over from an earlier call, a failed step or another model.
 *
 * Set-up: msm_model_create looks up the array's device address
 * (cudaGetSymbolAddress, with the model's device current), which loads the code
 * module that holds the array and so gives the array its device memory then, at
 * creation, not at the first call; the calls themselves do no set-up.
 *
 * Concurrency: the scratch is one array per device.  Calls that overlap on the
 * device (from other threads, or on other streams of the same device before the
 * previous call's work has finished) race on it and give wrong results.
 * Serialise them, e.g. by issuing them on one stream.
 *
 * Device-side failures are reported by the next msm_sync(), as for
 * msm_verify_step.
 */
#define MSM_NOALLOC_SCRATCH_BYTES (10u << 20)
msm_status msm_verify_step_noalloc(msm_model* model, const void* hidden_in, const int32_t* parent,
                                   int32_t pos0, void* const* k_cache, void* const* v_cache,
                                   float* logits_out, void* hidden_out, void* stream);

/* Wait for `stream`, then return (and clear) the device status latched by the
 * model's launches.  After MSM_ERR_DEVICE_TIMEOUT the model re-arms its exchange
 * buffers, so the next step starts clean. */
msm_status msm_sync(msm_model* model, void* stream);

/* Routing of the last completed step: idx int32 [n_layers][16][top_k] (expert
 * indices, larger logit first, ties to the lower index) and w fp32
 * [n_layers][16][top_k] (softmax over the selected logits).  Host buffers; either
 * may be NULL.  Synchronises the device. */
msm_status msm_get_routing(msm_model* model, int32_t* idx, float* w);

/* Tree as computed on the device in the last step: anc uint32 [16]
 * (ancestor-or-self bitmask), tpos int32 [16] (pos0 + depth).  Host buffers. */
msm_status msm_get_tree(msm_model* model, uint32_t* anc, int32_t* tpos);

/* Self-timing stamps of the last step (MSM_FLAG_SELF_TIMING):
 * uint64 [n_layers][grid_blocks][MSM_TIMING_EVENTS] %globaltimer values (ns), 0
 * where an event did not occur.  Event ids (per block of a launch; "_IN" = the
 * phase's input has been received and staged):
 *   0 start, 1 prologue in, 2 prologue done, 3 attention in, 4 attention done,
 *   5 split merge done, 6 o_proj in, 7 o_proj done, 8 pooler in, 9 pooler done,
 *   10 router in, 11 router done, 12 top-k done, 13 routing done, 14 GEMM1 done,
 *   15 GEMM2 in, 16 GEMM2 done, 17 combine done, 18 unpooler in, 19 unpooler done,
 *   20 tail in, 21 tail done, 22 end, 23 loader saw the routing, 24 loader done,
 *   25 expert dispatch built, 26 pooler input staged (before its norm), 27 first
 *   pooled row read for GEMM1, 28 / 29 first / second GEMM1 input row of the
 *   first compute warp staged, 30 pooler input normalised by the first compute
 *   warp, 31 pooler norm gain in shared memory; 32-39 o_proj units 0 and 1 of the block (first tile ready, last tile
 *   ready, partial sums stored, epilogue done), 40-43 GEMM1 of the first compute
 *   warp (first unit's tile ready / unit done, last unit's tile ready / done),
 *   44 / 45 loader issued the first / last o_proj tile, 46 / 47 the first / last
 *   GEMM1 tile; 48-51 GEMM2 of the first compute warp pair (first unit's tile ready
 *   / unit done, last unit's tile ready / done), 52 / 53 second GEMM2 staging
 *   round (experts 3-4 of a block; two per round) begun / done, 54 loader issued the first tile of the
 *   block's second o_proj unit; 55-62 the block's poller saw the phase-completion
 *   counter that releases the split merge, o_proj, pooler, router, top-k, combine,
 *   unpooler and tail reach the grid size.
 * `n` is the capacity of `buf` in elements. */
#define MSM_TIMING_EVENTS 192
msm_status msm_get_timing(msm_model* model, uint64_t* buf, size_t n);

msm_status msm_get_stats(const msm_model* model, msm_stats* out);

/* Diagnostic: copy an exchange buffer of the last launch of the last step to host
 * memory.  `name` is one of "o" (attention output, bf16 [16][n_q_heads head_dim]),
 * "h1" (residual after attention, bf16 [16][d_model]), "u" (pooled, bf16
 * [16][pool_dim]), "logits" (router logits, fp32 [16][n_experts]), "a" (SwiGLU
 * activations, fp32 [16 top_k][ffn_dim]), "z" (combined expert output, bf16
 * [16][pool_dim]), "h2" (layer output, bf16 [16][d_model]).  Slots a launch never
 * filled keep their sentinels (0xFFFF / -0.0).  `bytes` is the capacity of `host`.
 * Synchronises the device. */
msm_status msm_get_exchange(msm_model* model, const char* name, void* host, size_t bytes);

/*
 * Accept step after a verify step: the target's greedy choice at each tree node,
 * the walk down the tree, and KV-cache compaction (alphasignal.ai, § "Draft and
 * verify share one graph": candidates the target agrees with become output
 * tokens, rejected branches are dropped; orcarouter.ai, closing figure: greedy
 * decoding, accept inside the step's CUDA graph).
 *   logits   device fp32 [16][vocab], the verify step's logits_out (read)
 *   tokens   host int32 [16]: the draft token of each tree node; tokens[0] (the
 *            root) is not checked; every id must lie in [0, vocab)
 *   parent   host int32 [16], the verify step's tree
 *   pos0, k_cache, v_cache   as passed to the verify step
 *   result   device int32 [MSM_ACCEPT_RESULT_INTS] (written):
 *            [0] a = number of accepted nodes, root included (1..16)
 *            [1] the bonus token: the greedy choice at the last accepted node
 *            [2 + j] path[j], the j-th accepted node (path[0] = 0), -1 for j >= a
 *            [18 + i] the greedy choice (argmax of the logits) at node i
 * Greedy choice: the largest logit, the smallest index among equal ones; a NaN
 * ranks above every number.  Walk: from the root, move to the child (smallest
 * tree index first) whose token is the current node's choice; stop when none is.
 * Compaction: for j < a, cache row pos0 + j of every layer, K and V, every KV head
 * receives row pos0 + path[j]; no other row is written.  Everything runs on the
 * device (two launches on `stream`, no host round trip), so a stream capture
 * records it.  It uses model-owned scratch (argmax partials, a ticket counter), so
 * accept calls of one model must not overlap on the GPU, like its steps.
 * Errors: MSM_ERR_UNSUPPORTED when vocab == 0, MSM_ERR_INVALID_ARG
 * for NULL or misaligned buffers, an invalid parent array, token ids or pos0;
 * nothing is enqueued then.
 */
#define MSM_ACCEPT_RESULT_INTS 34
msm_status msm_accept(msm_model* model, const float* logits, const int32_t* tokens, const int32_t* parent,
                      int32_t pos0, void* const* k_cache, void* const* v_cache, int32_t* result, void* stream);

/*
 * One CUDA graph per decode step (alphasignal.ai, § "Draft and verify share one
 * graph"; orcarouter.ai, closing figure): msm_graph_create captures the arming of
 * the model's exchange buffers, the verify step's n_layers launches, if
 * accept_result is not NULL msm_accept's launches, and a second arming (so eager
 * steps and replays may be mixed freely), and instantiates the graph.
 * Arguments are those of msm_verify_step and msm_accept; the tree, the tokens and
 * pos0 are recorded in the graph, as are all buffer addresses, so a replay reads
 * the buffers' current contents at those addresses.  msm_graph_launch replays it
 * on `stream`; every replay computes what the captured calls compute.
 * (msm_graph_create_dev below records a device-resident state instead of the tree,
 * tokens and pos0; msm_graph_create_spec adds the draft step and the embedding of
 * its proposal, so one graph holds the whole speculative step.)  The model must outlive its graphs;
 * replays of one model must not overlap on the GPU.  msm_graph_destroy frees the
 * graph (NULL is ignored).  Errors: those of the captured calls (nothing is
 * recorded then), MSM_ERR_CUDA for a failed capture or instantiation.
 */
typedef struct msm_graph msm_graph;

/*
 * Device-resident step inputs, so that one graph can serve every decode step
 * (the pages' plugin replays one graph per step; orcarouter.ai, closing figure):
 * a device int32 [MSM_STEP_STATE_INTS] array
 *   [0] pos0, [1 + i] parent[i], [17 + i] the draft token of tree node i, [33] unused
 * read by the kernels when they run, not when the call is made.  The caller
 * writes it (for instance with cudaMemcpyAsync on the same stream) before each
 * step.  The kernels check it (parent[0] == -1, 0 <= parent[i] < i, token ids in
 * [0, vocab), 0 <= pos0 <= max_ctx - 16); an invalid state makes every launch of
 * the step give up at entry without touching the caches or outputs, and the next
 * msm_sync() returns MSM_ERR_INVALID_ARG (msm_accept_dev then also writes a = 0
 * and -1 elsewhere in `result`).
 *   msm_verify_step_dev  = msm_verify_step with the tree and pos0 from `state`
 *   msm_accept_dev       = msm_accept with tree, tokens and pos0 from `state`
 *   msm_graph_create_dev = msm_graph_create capturing those two: a replay reads the
 *                          state's current contents, so one graph serves any tree
 *                          and position
 * Host errors as for the host-parameter calls, plus MSM_ERR_INVALID_ARG for a NULL
 * or misaligned state.
 */
#define MSM_STEP_STATE_INTS 34
msm_status msm_verify_step_dev(msm_model* model, const void* hidden_in, const int32_t* state, void* const* k_cache,
                               void* const* v_cache, float* logits_out, void* hidden_out, void* stream);
msm_status msm_accept_dev(msm_model* model, const float* logits, const int32_t* state, void* const* k_cache,
                          void* const* v_cache, int32_t* result, void* stream);
msm_status msm_graph_create_dev(msm_model* model, const void* hidden_in, const int32_t* state, void* const* k_cache,
                                void* const* v_cache, float* logits_out, void* hidden_out, int32_t* accept_result,
                                msm_graph** out);

msm_status msm_graph_create(msm_model* model, const void* hidden_in, const int32_t* parent, const int32_t* tokens,
                            int32_t pos0, void* const* k_cache, void* const* v_cache, float* logits_out,
                            void* hidden_out, int32_t* accept_result, msm_graph** out);
msm_status msm_graph_launch(msm_graph* graph, void* stream);
void msm_graph_destroy(msm_graph* graph);

/*
 * msm_draft_step: one pass of the draft model (a model created with
 * MSM_FLAG_DRAFT) over a block of 16 slots, proposing 15 tokens at once
 * (alphasignal.ai, § "Draft and verify share one graph": a 5-layer draft, one
 * launch per layer, its 15 candidates from one pass).  The pages give only the
 * widths; the layer follows the target layer's conventions:
 *   slot i sits at position pos0 + i (RoPE) and writes its K/V rows to cache row
 *   pos0 + i; it attends to every history row [0, pos0) and to all 16 slots;
 *   h1 = bf16(h + bf16(attn W_o^T)); z = bf16(silu(x W_gate^T) * (x W_up^T)) with
 *   x = RMSNorm(h1); h2 = bf16(h1 + bf16(z W_down^T)); after the last layer the
 *   final RMSNorm and the LM head give fp32 logits.
 *   hidden_in  device bf16 [16][d_model]: the block's input rows
 *   pos0       first cache row of the block: 0 <= pos0 <= max_ctx - 16
 *   k_cache / v_cache  host arrays of n_layers device pointers, bf16
 *              [n_kv_heads][max_ctx][head_dim] each (the draft's own caches)
 *   logits_out device fp32 [16][vocab] (required)
 *   tokens_out device int32 [16]: tokens_out[0] = -1 (slot 0 holds the caller's
 *              known token), tokens_out[i] = the argmax of slot i's logits (the
 *              smallest index among equal maxima): the proposal for position
 *              pos0 + i.  The proposal is a chain, parent[i] = i - 1.
 * Launches n_layers layer-kernel launches and two reduction launches on `stream`;
 * returns after enqueueing.  Errors: MSM_ERR_INVALID_ARG (NULL pointer, pos0 out
 * of range, model not a draft model); a failing launch reports at msm_sync.
 */
msm_status msm_draft_step(msm_model* draft, const void* hidden_in, int32_t pos0, void* const* k_cache,
                          void* const* v_cache, float* logits_out, int32_t* tokens_out, void* stream);

/*
 * msm_draft_step_dev: msm_draft_step with pos0 read from a device-resident step
 * state (MSM_STEP_STATE_INTS ints, as for msm_verify_step_dev) when the kernels run;
 * the proposal goes into the state: parent[i] = i - 1 (the chain) for every i, and
 * the token of node i = the argmax of slot i for i = 1..15.  The root's token
 * (state[17]) is the caller's and is not written.  An invalid pos0 makes the layer
 * launches give up at entry (msm_sync then returns MSM_ERR_INVALID_ARG); the state
 * is still written, from whatever logits_out held.
 */
msm_status msm_draft_step_dev(msm_model* draft, const void* hidden_in, int32_t* state, void* const* k_cache,
                              void* const* v_cache, float* logits_out, void* stream);

/*
 * msm_embed_dev: the verify step's input rows from an embedding table, read from a
 * step state when the kernel runs: hidden_out[i] = table[state[17 + i]] (the token
 * of tree node i).  The verify step takes its 16 input rows as given (the embedding
 * precedes it in the pages' decoder); this call lets one graph go from the draft's
 * proposal to the verify step's input without a host round trip.
 *   model      the target model (vocab > 0; its d_model and vocab size the table)
 *   table      device bf16 [vocab][d_model], caller-owned, 16-byte aligned
 *   hidden_out device bf16 [16][d_model], 16-byte aligned
 * One launch of 16 blocks on `stream`.  A token id outside [0, vocab) gives a zero
 * row and MSM_ERR_INVALID_ARG at the next msm_sync (the verify step's own state
 * check rejects the step then).  Host errors: MSM_ERR_INVALID_ARG (NULL or
 * misaligned pointers), MSM_ERR_UNSUPPORTED (vocab == 0).
 */
msm_status msm_embed_dev(msm_model* model, const void* table, const int32_t* state, void* hidden_out, void* stream);

/*
 * msm_graph_create_spec: one CUDA graph holding a whole speculative decode step on
 * a device-resident state (alphasignal.ai, § "Draft and verify share one graph"):
 *   msm_draft_step_dev(draft, draft_hidden_in, state, draft caches, draft_logits)
 *   msm_embed_dev(target, embed_table, state, hidden_buf)
 *   msm_verify_step_dev(target, hidden_buf, state, k_cache, v_cache, logits_out)
 *   msm_accept_dev(target, logits_out, state, k_cache, v_cache, accept_result)
 * with both models' exchange buffers armed before and after.  Before each replay
 * the caller sets state[0] (pos0) and state[17] (the root token, e.g. the previous
 * step's bonus token) and fills draft_hidden_in; the graph writes the rest of the
 * state, hidden_buf, both logits and accept_result.  Both models must be on one
 * device and outlive the graph; replays must not overlap.  Errors: those of the
 * captured calls, MSM_ERR_INVALID_ARG for a NULL draft, table, hidden_buf, state or
 * accept_result or models on different devices.
 */
msm_status msm_graph_create_spec(msm_model* target, msm_model* draft, const void* draft_hidden_in,
                                 void* const* draft_k_cache, void* const* draft_v_cache, float* draft_logits,
                                 const void* embed_table, void* hidden_buf, int32_t* state, void* const* k_cache,
                                 void* const* v_cache, float* logits_out, int32_t* accept_result, msm_graph** out);

/*
 * Paged KV cache: the K/V rows of many sequences in fixed-size pages of one pool per
 * layer, with the calls a serving loop makes around msm_verify_step and
 * msm_draft_step for prompts, batches and searches.  (The pages that describe the
 * verify step keep one user's contiguous caches; they describe none of this.)
 *
 * Layouts
 *   pool (layer)   16-bit floats [n_pages][n_kv_heads][page_rows][head_dim], K and V.
 *                  A page has the layout of a verify-step cache of page_rows rows: with
 *                  page_rows = max_ctx, page p of a layer's pools can be passed to
 *                  msm_verify_step as that layer's caches.
 *   table          int32 [n_seqs][max_pages]: the pages of each sequence in order;
 *                  -1 behind its last page
 *   lens           int32 [n_seqs]: rows of each sequence (0: an unused slot)
 *   refs           int32 [n_pages]: how many sequences hold the page; 0: free
 *   status         int32 [1]: 0, or what msm_pages_sync makes of it: the first error that
 *                  a kernel met
 *   scratch        int32 [msm_pages_scratch_ints(n_pages, n_seqs)], contents of no
 *                  interest between calls
 * Row r of sequence s is row r % page_rows of page table[s][r / page_rows].  All of
 * these are device buffers of the caller.  An empty cache has lens, refs and status
 * zero and table -1.
 *
 * resize, fork and compact change table, lens and refs on the device, in stream order
 * and without a host round trip, so a stream capture records them.  Their results do
 * not depend on timing: pages are always taken in the order of their index, the lowest
 * free one first.  Each of them either does what it was asked or, when it finds an
 * error (below), changes nothing and leaves the error in status.  From a resize or fork that
 * was not done until msm_pages_sync has returned the error, no call changes the cache:
 * resize, fork, compact and msm_pages_write do nothing (the lengths are not those
 * that they were made for; the rows of a write would replace the last ones that are
 * there), and msm_paged_attention reads the sequences as they stand.  Calls on one cache
 * must be ordered (one stream, or events); msm_pages_write and msm_paged_attention of
 * different layers may overlap each other.
 *
 * Errors met on the device are reported by msm_pages_sync: MSM_ERR_OOM (no free page
 * left), MSM_ERR_INVALID_ARG (values out of range).  Kernels never follow a page index
 * outside [0, n_pages).  Host errors of every call: MSM_ERR_INVALID_ARG (NULL or
 * misaligned pointers, sizes below 1, strides that are no multiple of 8 elements),
 * MSM_ERR_UNSUPPORTED (head_dim other than 64 or 128, n_q_heads / n_kv_heads other
 * than 1, 2, 4 or 8, more than 65535 kv heads, 2^31 or more table entries, 2^32 or more rows in a pool);
 * nothing is enqueued then.  The calls leave the current device as it was.
 */
typedef enum { MSM_BF16 = 0, MSM_FP16 = 1, MSM_E4M3 = 2, MSM_FP32 = 3 } msm_dtype;

typedef struct {
  int device;
  int dtype;                   /* MSM_BF16 or MSM_FP16: the pools, and the rows and queries used with them */
  int n_layers, n_pages, page_rows, n_kv_heads, head_dim;
  int n_seqs, max_pages;       /* rows and columns of the table */
  void* const* k_pages;        /* host arrays [n_layers] of device pointers, 16-byte aligned */
  void* const* v_pages;
  int32_t *table, *lens, *refs, *status, *scratch;
} msm_pages;

/* int32 entries of msm_pages.scratch (0 for sizes below 1) */
size_t msm_pages_scratch_ints(int n_pages, int n_seqs);

/*
 * New lengths for the sequences: new_lens device int32 [n_seqs], -1 = leave as it is.
 * A sequence that grows gets the pages it lacks from those free before the call, in
 * the order of the sequences; if it ends inside a page that other sequences hold too,
 * it first gets its own copy of that page's rows in every layer.  A sequence that
 * shrinks gives back the pages behind its new end (their table entries become -1);
 * length 0 frees it.  Rows that become part of a sequence hold what their pages held.
 * Device errors: MSM_ERR_OOM; MSM_ERR_INVALID_ARG for a length below -1 or above
 * max_pages * page_rows, or for tables that hold a page outside the pool.
 */
msm_status msm_pages_resize(const msm_pages* pages, const int32_t* new_lens, void* stream);

/*
 * Sequences that begin as another one stands: parent device int32 [n_seqs], -1 = none.
 * Sequence s with parent[s] = p gets p's length and shares all of its pages; both may
 * then be resized and written as if each had its own.  Device error:
 * MSM_ERR_INVALID_ARG if a parent is out of range, is s itself or has a parent in this
 * call, or if s is not empty.
 */
msm_status msm_pages_fork(const msm_pages* pages, const int32_t* parent, void* stream);

/*
 * The pages in use moved to the front of the pool in every layer: with n of them in
 * use, those at index n and above take the free indices below n, both in ascending
 * order, and the tables follow.  refs of the moved pages move with them.
 */
msm_status msm_pages_compact(const msm_pages* pages, void* stream);

/*
 * K/V rows of new tokens into one layer's pages.  The tokens of sequence s are rows
 * starts[s] .. starts[s + 1] - 1 of k and v; they become the last rows of the
 * sequence, which msm_pages_resize must have made room for.
 *   k, v    device [n_tokens][n_kv_heads][head_dim], strides in elements between
 *           tokens and between heads (multiples of 8), 16-byte aligned
 *   starts  device int32 [n_seqs + 1], ascending from 0; tokens at or behind
 *           starts[n_seqs] are ignored
 * Device error: MSM_ERR_INVALID_ARG for a token without a row, or whose page is free
 * or shared; that token is left out (the others are stored, and later calls too).
 */
msm_status msm_pages_write(const msm_pages* pages, int layer, const void* k, const void* v, int64_t k_token_stride,
                           int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t* starts, int n_tokens, void* stream);

/*
 * Attention of one new token per sequence over one layer's pages (plain decoding):
 *   out[s][h] = sum_r softmax_r(scale q[s][h] . k_r) v_r   over the rows r of sequence s,
 * query head h reading kv head h / (n_q_heads / n_kv_heads).  The new token is the
 * sequence's last row (written before the call); with window > 0 it sees the last
 * `window` rows only, as on the verify step's sliding-window layers.  A sequence
 * without rows gives zeros.  Rows behind a sequence's end or before its window are not
 * read, whatever they hold.  32-bit scores and sums; for their product with v the weights
 * are two 16-bit terms (off by at most 3 x 2^-16 of themselves, fp16 3 x 2^-22).
 *   q, out     device [n_seqs][n_q_heads][head_dim], strides in elements between
 *              sequences and between heads (multiples of 8), 16-byte aligned
 *   workspace  device buffer of msm_paged_attention_workspace bytes (0: an argument is
 *              wrong, see msm_last_error), 16-byte aligned.  It must be zero before its
 *              first call; a call leaves its counters zero for the next one.  Calls that
 *              share a workspace must not overlap on the GPU (neither must graphs that
 *              recorded them), and must have the same n_q_heads, n_kv_heads and head_dim.
 * Device error: MSM_ERR_INVALID_ARG for a row on a page outside the pool; such rows are
 * left out (a sequence of which no row is left gives zeros).
 */
size_t msm_paged_attention_workspace(const msm_pages* pages, int n_q_heads);
msm_status msm_paged_attention(const msm_pages* pages, int layer, const void* q, int64_t q_seq_stride,
                               int64_t q_head_stride, int n_q_heads, float scale, int window, void* out,
                               int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * msm_paged_attention with sinks: on a sliding-window layer (window > 0) the first `sinks` rows of a
 * sequence stay visible behind the window, row r of n being seen if n - 1 - r < window or
 * r < sinks.  Without a window every row is seen anyway.  Rows between the sinks and the window are
 * not read.  Workspace, errors and arithmetic are those of msm_paged_attention, which is this
 * call with sinks = 0; a negative number of sinks is MSM_ERR_INVALID_ARG.
 */
msm_status msm_paged_attention_sinks(const msm_pages* pages, int layer, const void* q, int64_t q_seq_stride,
                                     int64_t q_head_stride, int n_q_heads, float scale, int window, int sinks,
                                     void* out, int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Wait for `stream`, then return (and clear) the device status of the cache. */
msm_status msm_pages_sync(const msm_pages* pages, void* stream);

/*
 * Paged KV cache in 8 bits: the pools hold e4m3 codes, and every block of block_rows rows of one
 * page and head has a 32-bit scale, K and V apart.  Row r of a page belongs to block r / block_rows of
 * the page; where block_rows does not divide page_rows the page's last block is shorter.  A value is
 * code x scale.
 *   pages      as for a cache of 16 bits, with dtype = MSM_E4M3 and pools e4m3
 *              [n_pages][n_kv_heads][page_rows][head_dim]
 *   block_rows 1 .. page_rows
 *   k_scales, v_scales  host arrays [n_layers] of device pointers, fp32
 *              [n_pages][n_kv_heads][ceil(page_rows / block_rows)], finite and not negative (0: the block's
 *              values are 0)
 * Tables, errors and the order of calls are those of the calls on msm_pages; the calls that move rows
 * move their scales too.
 */
typedef struct {
  msm_pages pages;
  int block_rows;
  float* const* k_scales;
  float* const* v_scales;
} msm_qpages;

msm_status msm_qpages_resize(const msm_qpages* pages, const int32_t* new_lens, void* stream);
msm_status msm_qpages_fork(const msm_qpages* pages, const int32_t* parent, void* stream);
msm_status msm_qpages_compact(const msm_qpages* pages, void* stream);
msm_status msm_qpages_sync(const msm_qpages* pages, void* stream);

/*
 * msm_pages_write into 8 bits: k and v hold dtype (MSM_BF16 or MSM_FP16) elements.  For each head and block
 * of rows, with amax the largest finite magnitude among the block's new rows, the least power of two s >= 2^-126
 * with amax <= 448 s (0 for amax = 0) is what they need.  A block whose first row is new takes it as its scale.
 * In one that begins with older rows of the sequence the scale becomes the larger of it and the old one,
 * and where that is larger than the old one the older codes are multiplied by old / new in 32 bits and rounded
 * again.  New elements are divided by the scale and rounded to nearest even, infinities to +-448 (in a block of
 * scale 0, too, where their value is 0), NaN stays NaN.  (Between powers of two the older codes lose bits below 2^-6 of
 * the scale only.)
 */
msm_status msm_qpages_write(const msm_qpages* pages, int layer, int dtype, const void* k, const void* v,
                            int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                            int64_t v_head_stride, const int32_t* starts, int n_tokens, void* stream);

/*
 * msm_paged_attention_sinks over a cache in 8 bits; q and out hold dtype (MSM_BF16 or MSM_FP16) elements.
 * The codes are exact in the products with q and the weights, 16-bit floats (fp16, the head's q scaled by a power of
 * two); scores and sums have 32 bits, and a weight times V's scale is two 16-bit terms (off by at most
 * 3 x 2^-22 of itself or 2^-39 of the largest).
 */
size_t msm_qpages_attention_workspace(const msm_qpages* pages, int n_q_heads);
msm_status msm_qpages_attention(const msm_qpages* pages, int layer, int dtype, const void* q, int64_t q_seq_stride,
                                int64_t q_head_stride, int n_q_heads, float scale, int window, int sinks, void* out,
                                int64_t out_seq_stride, int64_t out_head_stride, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Causal attention of whole prompts, packed one behind the other: the pass that fills
 * the caches which the verify step, the draft step and msm_paged_attention read.
 * Sequence s has the queries q_starts[s] .. q_starts[s + 1] - 1 and the keys k_starts[s]
 * .. k_starts[s + 1] - 1, aligned at their ends: with nq queries and nk keys, query i
 * sees the keys j with 0 <= i + (nk - nq) - j, and with window > 0 only those with
 * i + (nk - nq) - j < window (the verify step's sliding window).  nk > nq resumes a
 * prompt whose first rows are cached already; a query that sees no key gives zeros.
 *   out[i][h] = sum_j softmax_j(scale q[i][h] . k[j]) v[j]
 * with kv head h / (n_q_heads / n_kv_heads).  32-bit scores and sums; the weights are
 * rounded to the 16-bit type for their product with v (fp16: to 0 below 2^-28 of the
 * largest).  Keys that a query does not see have no part in its result, whatever they hold.
 *   q, out   device [n_q][n_q_heads][head_dim]; k, v device [n_k][n_kv_heads][head_dim]:
 *            strides in elements between tokens and between heads (multiples of 8, at
 *            least head_dim, below 2^31), 16-byte aligned.  A verify-step cache is read in
 *            place with token stride head_dim and head stride max_ctx * head_dim.  out must not
 *            overlap the inputs.
 *   q_starts, k_starts  device int32 [n_seqs + 1], ascending from 0, at most n_q and n_k
 *            (larger values are cut off there); rows of out at or behind
 *            q_starts[n_seqs] are left as they are.  A sequence without queries stands for
 *            keys to be passed over, as the rows that a cache has to spare.  n_q = 0 does
 *            nothing; with n_k = 0 k and v may be NULL.
 * Host errors: MSM_ERR_INVALID_ARG (NULL or misaligned pointers, sizes out of range,
 * strides), MSM_ERR_UNSUPPORTED (head_dim other than 64 or 128, n_q_heads / n_kv_heads
 * other than 1, 2, 4 or 8, more than 65535 kv heads, n_q or n_k of 2^27 or more, or
 * (n_seqs + n_q * n_q_heads / n_kv_heads / 256) * n_kv_heads of about 2^31 or more).
 * Bounded waits: every wait inside the kernel gives up after 2 s on the clock (a GPU that
 * does other work meanwhile counts towards it) and lets the launch finish; the rows of that
 * block that were not done are NaN then, and *status, where it is not NULL and holds 0, becomes
 * MSM_ERR_DEVICE_TIMEOUT.  Nothing clears it but the caller.
 */
typedef struct {
  int device;
  int dtype;  /* msm_dtype */
  int n_seqs, n_q, n_k, n_q_heads, n_kv_heads, head_dim;
  int window; /* 0: every key up to the query's own position */
  float scale;
  const void *q, *k, *v;
  void* out;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
      out_token_stride, out_head_stride;
  const int32_t *q_starts, *k_starts;
  int32_t* status;  /* device int32 [1], or NULL */
  uint32_t flags;   /* MSM_FLAG_TEST_DROP_HANDOFF (no key or value is loaded, so that the waits run out), or 0 */
} msm_prompt;
msm_status msm_prompt_attention(const msm_prompt* prompt, void* stream);

/*
 * msm_prompt_attention with sinks: with window > 0 the first `sinks` keys of a sequence stay visible
 * behind the window, key j being seen by the query at position i' = i + (nk - nq) if j <= i' and
 * (i' - j < window or j < sinks).  msm_prompt_attention is this call with sinks = 0; a negative number
 * of sinks is MSM_ERR_INVALID_ARG.
 */
msm_status msm_prompt_attention_sinks(const msm_prompt* prompt, int sinks, void* stream);

/*
 * Drawing one token per row of logits, from given random numbers: the step from the LM head's logits
 * (those of msm_verify_step and msm_draft_step among them) to the next tokens where msm_accept's greedy
 * choice is not wanted.  With x a row, M its maximum, T its temperature and w_i = exp((x_i - M) / T):
 *   - the tokens are ordered by x, the larger first, among equals the lower index first; -inf and NaN are
 *     never drawn;
 *   - top_k > 0 keeps the first top_k of them;
 *   - top_p < 1 keeps of these the shortest beginning whose weights add up to at least top_p times theirs
 *     (at least one token);
 *   - min_p keeps of these the ones with w >= min_p;
 *   - the token is the lowest index whose weight, added to those of the kept lower indices, exceeds
 *     random x the sum over all that are kept (random = 1: the last one that has a weight).
 * T = 0 takes the largest logit (the lowest index among equals).  In a row with logits of +inf these alone
 * can be drawn, with equal weights.  Weights are held as multiples of 2^-42 (of the largest; min_p is at least that),
 * so sums are exact and do not depend on timing: each is off by at most 1.1 x 2^-30 of itself and 2^-43 of the
 * largest, so that small ones keep few bits, and a border or a number that is nearer to a sum than these errors add up to
 * may fall to its other side.  (With logits or temperatures beyond 2^110 they have 32-bit floating point's precision, and
 * differences of logits beyond its largest number count as infinite; temperatures between 0 and 2^-127 count as about that.)
 *   logits     device MSM_FP32, MSM_BF16 or MSM_FP16 [n_rows][vocab], row_stride elements between rows (0:
 *              every row is the same one), aligned to their type
 *   temperature, top_k, top_p, min_p  device [n_rows], fp32 and int32, or NULL for 1, 0 (no limit), 1 and 0
 *   random     device fp32 [n_rows], 0 .. 1
 *   tokens     device int32 [n_rows]: the tokens; -1 for a row without a token that can be drawn, and for one
 *              whose temperature is negative or not finite, or whose top_p, min_p or random is outside 0 .. 1
 *   probs      device fp32 [n_rows] or NULL: the token's probability among those kept (0 beside -1), computed in 32
 *              bits (off by at most 2^-20 of itself)
 *   kept       device int32 [n_rows] or NULL: how many tokens are kept (0 beside -1)
 * Host errors: MSM_ERR_INVALID_ARG (NULL or misaligned pointers, sizes below 1 - n_rows = 0 does nothing -,
 * a negative stride, another dtype), MSM_ERR_UNSUPPORTED (vocab above 2^20, 2^24 rows or more).
 * One launch, no workspace; the logits are read once up to about 400,000 (MSM_FP32) or 800,000 of them.
 */
typedef struct {
  int device;
  int dtype; /* msm_dtype of the logits */
  int n_rows, vocab;
  const void* logits;
  int64_t row_stride;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *random;
  int32_t* tokens;
  float* probs;
  int32_t* kept;
} msm_sampling;
msm_status msm_sample(const msm_sampling* sampling, void* stream);

/* Message of the last error on the calling thread ("" if none). */
const char* msm_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MSM_H */
