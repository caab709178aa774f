/*
 * medusa.h -- C ABI of the Medusa draft-and-verify decode step on one GPU (sm_103a).
 *
 * One call of medusa_step() performs a full decode step for B independent sequences:
 *   (1) the K residual SiLU heads and the LM head on the last hidden state h_t, with a
 *       top-s_k per head and the greedy root token,
 *   (2) the packed candidate tree (tokens, depth position ids, ancestor bitmask, paths),
 *   (3) tree attention of every node over the KV prefix plus its own ancestors, through
 *       one synthetic attention layer standing in for the backbone,
 *   (4) verification logits, greedy or typical acceptance, longest accepted path,
 *   (5) KV-cache compaction to the accepted path, and the carried state for the next step.
 * Sources (cited below by tag):
 *   [MEDUSA]  "Medusa: Simple LLM Inference Acceleration Framework with Multiple Decoding
 *             Heads" (structured summary of arXiv 2401.10774), Section 3.
 *   [NOTES]   "Accelerating LLM Inference with Speculative Decoding: Notes on Medusa".
 *   [READING] "MEDUSA 精读", sections 3, 4 and 6.
 *
 * Conventions (every entry point):
 *   - Pointers marked "device" are CUDA device pointers owned by the caller; "host" are
 *     host pointers owned by the caller.  The library allocates no device memory per call:
 *     scratch comes from the caller's workspace (medusa_workspace_size()).  Only
 *     medusa_plan_create() allocates (the uploaded tree spec and a status word) and
 *     medusa_plan_destroy() frees it.
 *   - Matrices are row-major [out][in]: a projection R^in -> R^out is stored out rows of
 *     in contiguous elements.  "dtype" elements are float (MEDUSA_F32) or bfloat16
 *     (MEDUSA_BF16) as the plan says; hidden states and every float output are float32.
 *   - `stream` is a cudaStream_t passed as void*.  Calls only enqueue work on it: they do
 *     not synchronise and may return before the GPU has finished.
 *   - Argument, shape and alignment errors are detected on the host before anything is
 *     launched and return MEDUSA_ERR_INVALID / MEDUSA_ERR_UNSUPPORTED.  Anomalies only the
 *     GPU can see (a KV length past capacity, a page id out of range, non-finite logits)
 *     set bits of the plan's device status word (MEDUSA_FLAG_*) and never trap; read them
 *     with medusa_get_status().  Launch failures return MEDUSA_ERR_CUDA.
 *   - Calls on one plan may run on different streams only if the caller orders them;
 *     concurrent calls must use distinct workspaces.
 */
#ifndef MEDUSA_H_
#define MEDUSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MEDUSA_MAX_HEADS 8     /* K <= 8 Medusa heads ([MEDUSA] §3.4: five suffice) */
#define MEDUSA_MAX_TOPS 16     /* s_k <= 16 candidates per head */
#define MEDUSA_MAX_NODES 256   /* N + 1 <= 256 packed tree nodes (root included) */
#define MEDUSA_MAX_LAYERS 1024 /* backbone layers of medusa_step_layers */
#define MEDUSA_MAX_CAPACITY (1 << 24) /* slots per sequence of a medusa_cache */

typedef enum {
  MEDUSA_OK = 0,
  MEDUSA_ERR_INVALID = -1,      /* bad argument, shape, tree spec or pointer alignment */
  MEDUSA_ERR_UNSUPPORTED = -2,  /* valid but outside the built kernels' limits */
  MEDUSA_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed */
  MEDUSA_ERR_DEVICE = -4,       /* medusa_get_status(): the device status word is set */
  MEDUSA_ERR_WORKSPACE = -6     /* workspace NULL or smaller than medusa_workspace_size */
} medusa_status;

enum { MEDUSA_F32 = 0, MEDUSA_BF16 = 1 };
enum { MEDUSA_KV4 = 2 };   /* a cache's format only: 4-bit blocks, see medusa_cache_dims */
enum { MEDUSA_GREEDY = 0, MEDUSA_TYPICAL = 1, MEDUSA_REJECT = 2 };

/* device status word bits */
#define MEDUSA_FLAG_TOKEN_RANGE 0x1u  /* a selected token id fell outside [0, V) */
#define MEDUSA_FLAG_KV_CAPACITY 0x2u  /* len + tree/path length would exceed capacity */
#define MEDUSA_FLAG_PAGE_RANGE  0x4u  /* a page-table entry fell outside [0, num_pages) */
#define MEDUSA_FLAG_NONFINITE   0x8u  /* a logit or softmax statistic was NaN or Inf */
#define MEDUSA_FLAG_TIMEOUT     0x10u /* a bounded wait in a pipelined kernel expired */
#define MEDUSA_FLAG_POS_RANGE   0x20u /* a position fell outside a rotary table */
#define MEDUSA_FLAG_ROW_RANGE   0x40u /* a row index, offset or count was out of range */

typedef struct medusa_plan medusa_plan;   /* opaque */

/* Model and batch sizes. */
typedef struct {
  int B;            /* sequences */
  int d;            /* hidden size */
  int V;            /* vocabulary */
  int K;            /* Medusa heads, 1..MEDUSA_MAX_HEADS */
  int Hq, Hkv, dh;  /* query heads, key/value heads (Hq % Hkv == 0), head dim */
  int dtype;        /* MEDUSA_F32 or MEDUSA_BF16: weights, embedding and KV cache */
  float rope_base;  /* rotary base (10000 for Llama) */
  int capacity;     /* KV slots per sequence */
  int page_size;    /* 0: contiguous cache; > 0: tokens per page */
  int num_pages;    /* paged cache: pages in the pool (bounds for page-table entries) */
} medusa_dims;

/* Packed candidate tree ([MEDUSA] §3.4 Tree Attention, Steps 1-2; [READING] section 6).
 * Node 0 is the root (the LM head's greedy token).  Node n >= 1 takes the rank[n]-th
 * best token of head depth(n); parent[n] < n.  depth(n) = depth(parent[n]) + 1 <= K. */
typedef struct {
  int K;                           /* heads the tree draws on */
  int s[MEDUSA_MAX_HEADS];         /* top-s_k per head, 1..MEDUSA_MAX_TOPS */
  int N;                           /* candidate nodes, root excluded */
  const int32_t* parent;           /* host [N+1], parent[0] = -1 */
  const int32_t* rank;             /* host [N+1], rank[0] = 0, rank[n] < s[depth(n)-1] */
} medusa_tree_spec;

/* Weights (device, dtype elements, row-major [out][in]). */
typedef struct {
  const void* w1;   /* [K][d][d]   head k's first projection ([MEDUSA] §3.4 head eq.) */
  const void* w2;   /* [K][V][d]   head k's vocabulary projection */
  const void* lm;   /* [V][d]      LM head */
  const void* emb;  /* [V][d]      token embedding of the synthetic layer */
  const void* wq;   /* [Hq*dh][d]  query projection */
  const void* wk;   /* [Hkv*dh][d] key projection */
  const void* wv;   /* [Hkv*dh][d] value projection */
  const void* wo;   /* [d][Hq*dh]  output projection */
} medusa_weights;

/* KV cache (device).  Contiguous: k, v each [B][capacity][Hkv][dh].  Paged: k, v each
 * [num_pages][page_size][Hkv][dh] and page_table [B][capacity/page_size]; slot t of
 * sequence b is row t % page_size of page page_table[b][t / page_size].  Keys are stored
 * after RoPE. */
typedef struct {
  void* k;
  void* v;
  const int32_t* page_table;  /* device, NULL for a contiguous cache */
  const int32_t* len;         /* device [B] prefix lengths at the start of the step */
  int32_t* len_out;           /* device [B] lengths after compaction (may alias len) */
} medusa_kv;

/* Acceptance rule ([MEDUSA] §3.4 Typical Acceptance Scheme and the speculative-decoding
 * rejection rule it replaces).
 *   MEDUSA_GREEDY   a candidate is kept iff it is its parent's greedy token.
 *   MEDUSA_TYPICAL  kept iff p(x) > min(eps, delta * exp(-H(p))), p = softmax(z / T).
 *   MEDUSA_REJECT   rejection sampling with the heads' top-s tokens as point-mass drafts:
 *                   from the root, the current node's children are tried in rank order,
 *                   child x kept iff u < p(x) / R (R = probability mass not yet rejected
 *                   at this node, 1 at first), else R -= p(x); the first kept child becomes
 *                   the current node.  Where no child is kept, the next step's root is
 *                   drawn from p at the current node without the rejected tokens (the
 *                   smallest token whose cumulative weight exceeds u_final times the
 *                   remaining total).  The emitted tokens are then distributed as p.
 *                   uniforms: device [B][1 + 16 K] floats in [0, 1): [b][0] = u_final,
 *                   [b][1 + 16 (d - 1) + j] = u of the j-th child tried at depth d.  A new
 *                   set is needed for every step, so the decode loop rejects this mode.
 * Temperature 0 is greedy in every mode. */
typedef struct {
  int mode;           /* MEDUSA_GREEDY, MEDUSA_TYPICAL or MEDUSA_REJECT */
  float temperature;  /* typical / reject: softmax temperature; 0 means greedy */
  float eps;          /* typical: hard threshold epsilon */
  float delta;        /* typical: entropy-threshold multiplier delta */
  const float* uniforms;  /* reject: see above; unused (may be NULL) otherwise */
} medusa_accept;

/* Step outputs (device). */
typedef struct {
  int32_t* out_tok;     /* [B][K+1] root then accepted tokens, -1 past n_acc */
  int32_t* n_acc;       /* [B] kept tokens = 1 + accepted candidates */
  int32_t* path_nodes;  /* [B][K+1] packed indices of the kept nodes, -1 padded */
  float* h_next;        /* [B][d] hidden state at the last kept node (next h_t) */
  int32_t* root_next;   /* [B] greedy token at the last kept node (next root) */
} medusa_outputs;

/* ------------------------------------------------------------------ plan */
/* Validates dims and the tree spec, uploads the spec and allocates the status word.
 * Returns MEDUSA_ERR_INVALID for inconsistent sizes or a malformed tree (parent >= own
 * index, depth > K, rank >= s), MEDUSA_ERR_UNSUPPORTED past the kernels' limits
 * (N+1 > 256, s_k > 16, K > 8, dh not in {32, 64, 128}, d or Hq*dh not a multiple
 * of 64 for bf16). */
medusa_status medusa_plan_create(const medusa_dims* dims, const medusa_tree_spec* tree,
                                 medusa_plan** out);
void medusa_plan_destroy(medusa_plan* plan);
/* Bytes of device workspace one medusa_step (or any stage call) needs. */
size_t medusa_workspace_size(const medusa_plan* plan);
/* Synchronises `stream`, returns the device status word in *flags and clears it.
 * MEDUSA_ERR_DEVICE when a flag was set, MEDUSA_OK otherwise. */
medusa_status medusa_get_status(const medusa_plan* plan, void* stream, uint32_t* flags);
/* Failure-path testing (the pages have no counterpart): the next verification-logit GEMM
 * this plan launches (in medusa_step, medusa_step_layers, medusa_verify_logits or a
 * decode loop captured after this call) has its MMA thread first wait, for at most `ns`
 * nanoseconds, on a barrier that nothing arrives on.  The wait runs out and the kernel
 * takes the path of a wait on a copy that never landed: it sets MEDUSA_FLAG_TIMEOUT,
 * lets its other waits run to their own ~1 s limits, drains its copies in flight, frees
 * its tensor memory and returns, so the call's outputs are meaningless but the CUDA
 * context stays usable.  One-shot: the setting is cleared when that GEMM is launched.
 * MEDUSA_ERR_INVALID for ns = 0 or above 10 s; MEDUSA_ERR_UNSUPPORTED for plans without
 * the tensor-core projections (fp32). */
medusa_status medusa_plan_expire_wait_once(medusa_plan* plan, unsigned long long ns);

/* ------------------------------------------------------------------ full step */
/* One decode step ([MEDUSA] §3.2 information flow, steps (2)-(6); [READING] section 3).
 * h: device [B][d] last hidden state.  root_in: device [B] first token carried from the
 * previous step's root_next, or NULL to take the LM head's greedy token on h.  With
 * root_in given the LM head is not applied to h (it would only yield the root), so a
 * step of the steady-state decode loop reads the LM head once, for verification.
 * out->h_next may alias h and out->root_next may alias root_in: both inputs are read
 * before the step writes its outputs. */
medusa_status medusa_step(const medusa_plan* plan, const float* h, const int32_t* root_in,
                          const medusa_weights* w, const medusa_kv* kv, medusa_accept acc,
                          const medusa_outputs* out, void* workspace, size_t ws_bytes,
                          void* stream);

/* ---- multi-layer backbone
 * The tree nodes pass through n synthetic layers instead of one, the way a real
 * backbone's per-layer calls would ([MEDUSA] §3.4 Tree Attention: every layer attends
 * over its own cache plus the tree under the same mask and position ids):
 *   x_0 = E[tok];  layer l: q, k, v = Wq_l x_l, Wk_l x_l, Wv_l x_l (RoPE at the node
 *   position), o_l = tree attention over layer l's prefix and the tree's layer-l keys,
 *   x_{l+1} = x_l + Wo_l o_l;  h' = x_n  (verification, acceptance and h_next as in
 *   medusa_step).  After acceptance the kept nodes' keys/values are appended to every
 *   layer's cache.
 * One medusa_layer per layer: its projections ([out][in] row-major, the plan's dtype,
 * 16-byte aligned; shapes as in medusa_weights) and its KV cache (the layout medusa_kv
 * describes; every layer shares the page table and the lengths). */
typedef struct {
  const void* wq;   /* [Hq*dh][d]  */
  const void* wk;   /* [Hkv*dh][d] */
  const void* wv;   /* [Hkv*dh][d] */
  const void* wo;   /* [d][Hq*dh]  */
  void* k;          /* this layer's cached keys   (device, caller-owned, updated) */
  void* v;          /* this layer's cached values (device, caller-owned, updated) */
} medusa_layer;

/* Bytes of workspace medusa_step_layers needs for n_layers layers (the single-layer size
 * plus each further layer's tree keys/values); 0 for n_layers outside 1..MEDUSA_MAX_LAYERS. */
size_t medusa_workspace_size_layers(const medusa_plan* plan, int n_layers);

/* One decode step through an n_layers-layer backbone.  h, root_in, acc, out, stream as
 * in medusa_step; w supplies the heads, the LM head and the embedding (its wq..wo are not
 * read); layers: host array of n_layers entries (read during the call only); kv supplies
 * the page table, len and len_out (its k, v are not read; len_out may alias len).
 * Errors: MEDUSA_ERR_INVALID for n_layers outside 1..MEDUSA_MAX_LAYERS, a NULL layer
 * pointer or misaligned weights, plus medusa_step's conditions.  With n_layers = 1 the
 * result equals medusa_step's with that layer's weights and cache. */
medusa_status medusa_step_layers(const medusa_plan* plan, const float* h, const int32_t* root_in,
                                 const medusa_weights* w, const medusa_layer* layers, int n_layers,
                                 const medusa_kv* kv, medusa_accept acc, const medusa_outputs* out,
                                 void* workspace, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ stages */
/* (a) Heads ([MEDUSA] §3.4 MEDUSA Heads eq.; Tree Attention Step 1).  Writes the
 * logits [B][K+1][V] (row 0: LM head, row k: head k) to `logits` (device, may be NULL to
 * keep them in the workspace; row 0 is left unwritten when root_in is given, as the LM
 * head pass is then skipped), topk_tok/topk_val [B][K][16] (ranks past s_k unspecified)
 * and root [B] (root_in's value when given, else the LM head's greedy token; ties to the
 * lowest token id). */
medusa_status medusa_heads(const medusa_plan* plan, const float* h, const int32_t* root_in,
                           const medusa_weights* w, float* logits, int32_t* topk_tok,
                           float* topk_val, int32_t* root, void* workspace, size_t ws_bytes,
                           void* stream);
/* (a') Heads stage without a workspace.  The paper has no counterpart to this: it is a
 * deployment aid for callers that cannot allocate device memory when they run the heads
 * (an engine that plans every buffer up front and forbids allocation while decoding, a
 * plug-in confined to another framework's memory pool, code that may run while the
 * stream is being captured into a CUDA graph).  It computes exactly what medusa_heads()
 * computes and writes the same topk_tok / topk_val / root outputs (the logits are not
 * returned).  Its scratch lives in one library-owned device array of
 * MEDUSA_NOALLOC_SCRATCH_BYTES, present on every GPU that loads the library until the
 * process exits; no cudaMalloc, cudaFree or other allocating call is made.
 *   - Like the step, it keeps no logits: the vocab projections keep each CTA's best
 *     candidates and a selection merges them.  Plans whose heads scratch exceeds the array
 *     (about B*(K+1)*slots*128 bytes of candidate lists, slots = V/128 from batch 2 and a
 *     few hundred at batch 1, plus B*K*d*8 bytes of head activations) get
 *     MEDUSA_ERR_UNSUPPORTED and nothing is launched.
 *   - The first call on a device looks up the array's address with that device current;
 *     make that first call before any stream capture begins.  The address is kept per
 *     device and context; the first call after a cudaDeviceReset looks it up again and
 *     must likewise come before any capture.
 *   - All calls share the array and it keeps the last call's contents (nothing in it
 *     needs to start at zero).  Calls whose GPU work overlaps race on it: order them on
 *     one stream. */
#define MEDUSA_NOALLOC_SCRATCH_BYTES (4u << 20)
medusa_status medusa_heads_noalloc(const medusa_plan* plan, const float* h, const int32_t* root_in,
                                   const medusa_weights* w, int32_t* topk_tok, float* topk_val,
                                   int32_t* root, void* stream);
/* (b) Tree build ([MEDUSA] §3.4 Tree Attention Steps 2-4; [READING] section 6).
 * tok [B][N+1] node tokens, pos [B][N+1] = len + depth, mask [N+1][8] uint32 ancestor
 * bitmask (bit j of word j/32 set iff node j is on the root->n path), retrieve [N+1][K+1]
 * packed root->leaf paths (leaves in packed order, -1 padded; rows past the path count
 * are -1).  topk_tok as written by medusa_heads. */
medusa_status medusa_tree_build(const medusa_plan* plan, const int32_t* topk_tok,
                                const int32_t* root, const int32_t* len, int32_t* tok,
                                int32_t* pos, uint32_t* mask, int32_t* retrieve, void* stream);
/* (c) Synthetic layer projections: x = E[tok]; q = Wq x, k = Wk x, v = Wv x per head;
 * rotate-half RoPE of q and k at pos ([MEDUSA] §3.4 Step 4).  q: [B][N+1][Hq][dh] float;
 * tree_k, tree_v: [B][N+1][Hkv][dh] dtype. */
medusa_status medusa_layer_qkv(const medusa_plan* plan, const medusa_weights* w,
                               const int32_t* tok, const int32_t* pos, float* q, void* tree_k,
                               void* tree_v, void* workspace, size_t ws_bytes, void* stream);
/* (d) Tree attention ([MEDUSA] §3.4 Tree Attention Steps 3 and 5): node n, query head h
 * attends to the prefix slots [0, len) of key/value head h/(Hq/Hkv) and to the tree keys
 * of its ancestors (mask).  o: [B][N+1][Hq][dh] float. */
medusa_status medusa_tree_attention(const medusa_plan* plan, const float* q,
                                    const medusa_kv* kv, const void* tree_k,
                                    const void* tree_v, const uint32_t* mask, float* o,
                                    void* workspace, size_t ws_bytes, void* stream);
/* (e) Synthetic layer output h' = E[tok] + Wo o.  hprime: [B][N+1][d] float. */
medusa_status medusa_layer_out(const medusa_plan* plan, const medusa_weights* w,
                               const int32_t* tok, const float* o, float* hprime,
                               void* workspace, size_t ws_bytes, void* stream);
/* (f) Verification logits z_n = LM h'_n ([MEDUSA] §3.4 Tree Attention Step 6) and, per
 * node row, the statistics acceptance needs: am [B][N+1] greedy token (lowest id on ties);
 * stats [B][N+1][4] = {max_v z/T, log sum_v exp(z/T - max), entropy H (nats), z_parent at
 * this node's token / T} (T = 1 when greedy; entry 3 of the root is 0).  logits: device
 * [B][N+1][V] or NULL to keep them in the workspace. */
medusa_status medusa_verify_logits(const medusa_plan* plan, const medusa_weights* w,
                                   const float* hprime, const int32_t* tok, medusa_accept acc,
                                   float* logits, int32_t* am, float* stats, void* workspace,
                                   size_t ws_bytes, void* stream);
/* (g) Acceptance ([MEDUSA] §3.4 Typical Acceptance Scheme, whole-candidate and first-token
 * handling): the root is kept; candidate c is accepted iff tok[c] == am[parent[c]]
 * (greedy, or typical at T = 0) or log p_parent(tok[c]) > min(log eps, log delta - H)
 * (typical).  The longest run of accepted nodes along a root->leaf path wins, ties to the
 * lowest path index.  MEDUSA_REJECT walks the tree instead (see medusa_accept) and draws
 * root_next from `logits` ([B][N+1][V], as written by medusa_verify_logits; required in that
 * mode, unused and may be NULL otherwise).  Writes every medusa_outputs field; h_next is
 * hprime at the last kept node and root_next its greedy token (or the draw). */
medusa_status medusa_verify(const medusa_plan* plan, const int32_t* tok, const int32_t* am,
                            const float* stats, const float* logits, const int32_t* retrieve,
                            const float* hprime, medusa_accept acc, const medusa_outputs* out,
                            void* stream);
/* (h) KV compaction ([READING] section 3: only the accepted path stays in the cache):
 * slots len .. len+n_acc-1 receive the tree keys/values of path_nodes; len_out = len +
 * n_acc.  Slots past capacity are not written and set MEDUSA_FLAG_KV_CAPACITY. */
medusa_status medusa_kv_compact(const medusa_plan* plan, const medusa_kv* kv,
                                const void* tree_k, const void* tree_v,
                                const int32_t* path_nodes, const int32_t* n_acc, void* stream);

/* ------------------------------------------------------------------ decode loop */
/* The steady-state decode loop ([MEDUSA] §3.2: every step's first token is the previous
 * step's greedy token at the last accepted node, and decoding continues from the hidden
 * state there).  medusa_loop_create() captures, once, one medusa_step whose state is
 * carried in place (root_in = root_next = root, h = h_next = h, kv->len_out == kv->len:
 * the cache grows by each step's kept tokens) followed by the bookkeeping that appends the
 * step's out_tok [B][K+1] and n_acc [B] to the caller's rings tokens [max_steps][B][K+1] and
 * n_acc [max_steps][B] (position: steps appended so far, modulo max_steps) as a CUDA graph;
 * medusa_loop_run() replays it n_steps times on `stream` (asynchronous).
 *   - h: device [B][d], root: device [B] (e.g. a first medusa_step's h_next and root_next);
 *     both hold the latest state after every step.
 *   - Every pointer given here (weights, cache, lengths, state, rings, workspace) is used by
 *     every replay: keep them allocated, and the plan alive, until medusa_loop_destroy().
 *   - The cache must have room for the steps to be run (len + K + 1 <= capacity at every
 *     step); past that MEDUSA_FLAG_KV_CAPACITY is set, as in medusa_step.
 *   - Creation allocates the loop's small device state (B*(K+2) ints and a counter) and
 *     captures on a private stream; it launches nothing.
 * medusa_loop_steps() synchronises `stream` and returns the number of steps appended. */
typedef struct medusa_loop medusa_loop;
medusa_status medusa_loop_create(const medusa_plan* plan, const medusa_weights* w,
                                 const medusa_kv* kv, medusa_accept acc, float* h, int32_t* root,
                                 int32_t* tokens, int32_t* n_acc, int max_steps, void* workspace,
                                 size_t ws_bytes, medusa_loop** out);
medusa_status medusa_loop_run(medusa_loop* loop, int n_steps, void* stream);
medusa_status medusa_loop_steps(const medusa_loop* loop, void* stream, long long* steps);
void medusa_loop_destroy(medusa_loop* loop);

/* ------------------------------------------------------------------ tracing */
/* Per-stage timing (CUDA events recorded on the launching stream around every stage the
 * following calls on this plan run; a stage is one kernel, or a projection and its split-K
 * summation pass).  medusa_profile_start() creates the events for up to max_launches stages
 * (host-side resource, no device memory); stages past that are not timed.
 * medusa_profile_stop() synchronises `stream`, aggregates by stage name into out (up to
 * max_kernels entries, in first-launch order), writes the entry count to *n and the number
 * of kernels the calling thread launched meanwhile (split-K passes included) to
 * *launches, and ends profiling.  Each call also appears as an NVTX range named after it. */
typedef struct {
  char name[32];
  int launches;
  double total_ms;
} medusa_kernel_time;
medusa_status medusa_profile_start(medusa_plan* plan, int max_launches);
medusa_status medusa_profile_stop(medusa_plan* plan, void* stream, medusa_kernel_time* out,
                                  int max_kernels, int* n, int* launches);

/* ------------------------------------------------------------------ host tree builders */
/* Cartesian tree of the per-head top-s_k ([MEDUSA] §3.4 Tree Attention Step 2) in
 * canonical packing (by depth, then rank path).  parent/rank: host arrays of at least
 * max_nodes entries.  Returns N+1 (nodes incl. the root) or a negative medusa_status. */
int medusa_tree_cartesian(int K, const int* s, int max_nodes, int32_t* parent, int32_t* rank);
/* Optimized tree ([MEDUSA] §3.4 Optimized Tree Construction; [NOTES] section 4): from
 * the root, repeatedly add the frontier node with the largest product of marginal
 * accuracies a[k*smax + i] along its path (ties to the smaller rank path) until N nodes;
 * canonical packing.  Returns N+1 or a negative medusa_status. */
int medusa_tree_greedy(int K, const int* s, int smax, const double* a, int N, int32_t* parent,
                       int32_t* rank);

/* ---- optimized tree on the device, and the tree size
 * The same construction as medusa_tree_greedy, on the GPU from a device table: one CTA
 * repeatedly takes the frontier node with the largest path product (formed root to leaf in
 * double precision, as the host builder forms it; ties to the smaller rank path) and adds
 * its children to the frontier, then packs the N chosen nodes canonically.
 *   a:        device [K][smax] doubles, a[k*smax + i] = head k+1's marginal accuracy at
 *             rank i (values in [0, 1]); s: host [K], 1 <= s[k] <= smax <= MEDUSA_MAX_TOPS
 *   N:        candidates, 1 <= N <= MEDUSA_MAX_NODES - 1 and at most the Cartesian tree's size
 *   parent, rank: device [N+1] outputs in canonical packing (parent[0] = -1, rank[0] = 0)
 *   expected: device [N+1] output or NULL: expected[n] = the expected number of accepted
 *             candidates of the tree of the first n nodes added (sum of their path
 *             products), so one call gives the curve for every size up to N
 * Asynchronous on `stream`.  MEDUSA_ERR_INVALID on a bad size or NULL pointer. */
medusa_status medusa_tree_greedy_device(int K, const int* s, int smax, const double* a, int N,
                                        int32_t* parent, int32_t* rank, double* expected,
                                        void* stream);
/* Tree size for the current batch and context ([MEDUSA] §6 Limitations and Trade-offs: the
 * best tree size depends on the context length; "Follow-Up Research": dynamic candidate
 * counts for batched inference): among n candidate sizes with measured (or modelled) step
 * times step_ms[i], the index maximising the expected tokens per unit time
 * (1 + expected[sizes[i]]) / step_ms[i], ties to the smaller size.  expected: host
 * [max_n + 1] as from medusa_tree_greedy_device.  Returns the index or a negative status. */
int medusa_tree_size_choose(const double* expected, int max_n, const int* sizes,
                            const double* step_ms, int n);

/* ------------------------------------------------------------------ rotary positions */
/* Rotation of query and key rows by their positions ([MEDUSA] §3.4 Step 4 uses the depth
 * positions medusa_tree_build writes), for callers whose checkpoints rotate differently from
 * medusa_layer_qkv's synthetic layer or whose rows come from another projection.
 *
 * Pair i < rot/2 of a head turns by the angle p * f_i at position p, with the plain
 * frequencies theta_i = base^(-2i/rot) and
 *   MEDUSA_ROPE_PLAIN   f_i = theta_i
 *   MEDUSA_ROPE_LINEAR  f_i = theta_i / factor
 *   MEDUSA_ROPE_BANDED  f_i = w_i theta_i + (1 - w_i) theta_i / factor with
 *                       w_i = clamp((turns_i - low) / (high - low), 0, 1), turns_i =
 *                       orig_pos theta_i / (2 pi): full turns over the original context
 *   MEDUSA_ROPE_RAMP    the same mixture, w_i falling linearly over the pair index, from 1
 *                       at a = max(0, floor(c(high))) to 0 at b = min(rot - 1, ceil(c(low)))
 *                       (clamped to [0, 1]; b - a taken as at least 0.001), where c(r) =
 *                       rot ln(orig_pos / (2 pi r)) / (2 ln base) is the index that makes r turns
 * Cosine and sine are multiplied by attn (0 means 1).  Layout MEDUSA_ROPE_HALF pairs element
 * i with i + rot/2, MEDUSA_ROPE_INTERLEAVED 2i with 2i + 1; elements past rot pass through:
 *   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin      (inverse: sin negated)
 * The table of cosines and sines is computed in double on the GPU when the handle is created,
 * rounded once to float; products and sums are single IEEE float operations, and the result
 * is rounded once to the rows' dtype. */
enum { MEDUSA_ROPE_HALF = 0, MEDUSA_ROPE_INTERLEAVED = 1 };
enum { MEDUSA_ROPE_PLAIN = 0, MEDUSA_ROPE_LINEAR = 1, MEDUSA_ROPE_BANDED = 2, MEDUSA_ROPE_RAMP = 3 };
typedef struct {
  int rot;         /* rotated elements of a head: even, >= 2 */
  int layout;      /* MEDUSA_ROPE_HALF or MEDUSA_ROPE_INTERLEAVED */
  int max_pos;     /* positions 0..max_pos-1; the table takes max_pos * rot floats */
  int scaling;     /* MEDUSA_ROPE_PLAIN .. MEDUSA_ROPE_RAMP */
  double base;     /* > 1 */
  double factor;   /* > 0; read unless PLAIN */
  double orig_pos; /* > 0; BANDED and RAMP */
  double low, high;/* turns, 0 < low < high; BANDED and RAMP */
  double attn;     /* multiplier of cosine and sine, 0 means 1 */
} medusa_rope_desc;
typedef struct medusa_rope medusa_rope;   /* opaque: the table and a status word, on one GPU */
/* Creates the handle on the current device (allocates, and waits for the table).  Destroying it frees
 * both, so it comes after every call has ended that was given the handle; a CUDA graph that captured
 * such calls keeps the addresses, and the handle has to stay until its last replay has ended. */
medusa_status medusa_rope_create(const medusa_rope_desc* desc, medusa_rope** out);
void medusa_rope_destroy(medusa_rope* rope);
/* As medusa_get_status, for the handle's own status word. */
medusa_status medusa_rope_get_status(const medusa_rope* rope, void* stream, uint32_t* flags);
/* One set of rows: element e of head h of row r is x[r * x_row + h * x_head + e] (strides in
 * elements), its result y[r * y_row + h * y_head + e]; no two results may share an element, here and in
 * the calls below (MEDUSA_ERR_INVALID).  y == x with equal strides turns the
 * rows in place; otherwise x and y must not overlap. */
typedef struct {
  const void* x;
  void* y;
  int heads;
  long long x_row, x_head, y_row, y_head;
} medusa_rope_rows;
/* Turns up to 4 sets of rows (queries, keys) in one launch.  dtype: MEDUSA_F32 or
 * MEDUSA_BF16 elements; dh >= rot elements per head; pos: device [rows].  A row whose position
 * is outside the table is passed through unturned and sets MEDUSA_FLAG_POS_RANGE.  rows = 0
 * does nothing.  Any alignment of whole elements works; rows whose pointers and strides are
 * multiples of 16 bytes (and rot/2 of 16 bytes for HALF, rot for INTERLEAVED) move in 16-byte
 * units, bf16 rows for which 8 bytes are such a multiple in 8-byte units. */
medusa_status medusa_rope_apply(const medusa_rope* rope, int dtype, int dh, int rows,
                                const int32_t* pos, const medusa_rope_rows* parts, int n_parts,
                                int inverse, void* stream);

/* ------------------------------------------------------------------ KV caches */
/* A cache of B sequences, contiguous or paged (the layouts medusa_kv describes), that these
 * calls fill, read back and attend over.  In the formats MEDUSA_F32 and MEDUSA_BF16 it is the
 * cache medusa_step works on.  MEDUSA_KV4 holds 4.5 bits an element: 16 consecutive slots of
 * one head are a block of 9 dh bytes,
 *   16 rows of dh/2 bytes: element 2i in the low, 2i + 1 in the high four bits of byte i
 *                          (e2m1: sign, and one of 0 .5 1 1.5 2 3 4 6),
 *   16 rows of dh/16 bytes: one e4m3 scale for each 16 elements,
 * and an element stands for e2m1 * e4m3 * g, g = k_scale for keys and v_scale for values (any
 * numbers from 1e-20 to 1e20 the caller keeps to; powers of two make every element exact in bf16).  The
 * blocks lie [B][Hkv][capacity/16] (contiguous) or [num_pages][Hkv][page_size/16] (paged), so
 * a head's blocks follow each other.  Writing takes, over each 16 elements, s = max|x| / (6 g)
 * rounded to e4m3 and each x / (g s) rounded to e2m1 (both to nearest, ties to even, the
 * largest where beyond); 16 elements that hold an infinity or a NaN read back as NaN and set
 * MEDUSA_FLAG_NONFINITE. */
typedef struct {
  int B;             /* sequences */
  int Hq, Hkv, dh;   /* query heads (a multiple of Hkv), key/value heads, head size 32, 64 or 128 */
  int format;        /* MEDUSA_F32, MEDUSA_BF16 or MEDUSA_KV4 */
  int capacity;      /* slots per sequence, at most MEDUSA_MAX_CAPACITY (paged: a multiple of page_size) */
  int page_size;     /* 0: contiguous; KV4: page_size, or the contiguous capacity, is a multiple of 16 */
  int num_pages;     /* paged: pages in the pool */
  int max_nodes;     /* query rows (tree nodes) per sequence and attention call, 1..MEDUSA_MAX_NODES */
} medusa_cache_dims;
/* opaque: sizes and a status word, on one GPU.  Calls, and graphs that captured them, keep the status
 * word's address: destroy the handle after the last of them has ended. */
typedef struct medusa_cache medusa_cache;
medusa_status medusa_cache_create(const medusa_cache_dims* dims, medusa_cache** out);
void medusa_cache_destroy(medusa_cache* cache);
/* Bytes of the key pool, and of the value pool. */
size_t medusa_cache_pool_bytes(const medusa_cache* cache);
/* Bytes of device workspace medusa_kv4_attention needs (256-byte aligned; 0 for other formats). */
size_t medusa_cache_workspace_size(const medusa_cache* cache);
/* As medusa_get_status, for the cache's own status word. */
medusa_status medusa_cache_get_status(const medusa_cache* cache, void* stream, uint32_t* flags);
/* Failure-path testing, as medusa_plan_expire_wait_once: in the next medusa_kv4_attention call on this
 * cache (a captured one: in every replay) a warp of each block first waits, for at most `ns` nanoseconds,
 * on a barrier that nothing arrives on, and then takes the path of a copy that never landed:
 * MEDUSA_FLAG_TIMEOUT is set, the other waits run to their ~1 s limits, and the call returns with a
 * meaningless o and a usable context.  MEDUSA_ERR_INVALID for ns = 0 or above 10 s,
 * MEDUSA_ERR_UNSUPPORTED for other formats. */
medusa_status medusa_cache_expire_wait_once(medusa_cache* cache, unsigned long long ns);

/* Rows for the cache.  k, v: element e of head h of row r at [r * row + h * head + e] (strides
 * in elements; heads less than 2^31 bytes apart), outside the pools.  Items are the rows as they
 * are appended; `rows` is how many item places there are, and they belong to the sequences in
 * one of two ways:
 *   packed  start: device [B+1], ascending, items start[b] .. start[b+1]-1 are sequence b's;
 *           places before start[0] and from start[B] on belong to none and are skipped
 *   padded  start NULL: rows = B * per_seq, sequence b has the first count[b] (device [B],
 *           NULL: all) of the per_seq places from b * per_seq
 * Offsets outside 0..rows and counts outside 0..per_seq are taken as the nearer end and set
 * MEDUSA_FLAG_ROW_RANGE, and so do offsets that fall (len_out may then count slots that were not
 * written).
 * index (device [rows], NULL: item i is row i): item i of sequence b is row
 * b * index_rows + index[i], 0 <= index[i] < index_rows; items outside are skipped and set
 * MEDUSA_FLAG_ROW_RANGE.  With per_seq = K+1, count = n_acc, index = path_nodes, index_rows =
 * N+1 and k, v the tree's keys/values this is medusa_kv_compact for any format. */
typedef struct {
  const void* k;
  const void* v;
  int dtype;                            /* MEDUSA_F32 or MEDUSA_BF16 */
  long long k_row, k_head, v_row, v_head;
  int rows;
  const int32_t* start;
  int per_seq;
  const int32_t* count;
  const int32_t* index;
  int index_rows;
  const int32_t* pos;                   /* device [rows]: rotate item i as position pos[i] (NULL: its slot) */
} medusa_kv_rows;
/* Item j of sequence b goes to slot len[b] + j; its key is first turned by `rope` (NULL: as it
 * is).  len_out[b] = min(len[b] + items, capacity); it may alias len, and both lie apart from
 * everything else.  Slots past the capacity are not written and set MEDUSA_FLAG_KV_CAPACITY (as
 * a len outside 0..capacity does, which is then taken as the nearer end), a page outside the
 * pool MEDUSA_FLAG_PAGE_RANGE; an item with a position outside the table is stored unturned and
 * sets MEDUSA_FLAG_POS_RANGE.  No two sequences may share a page that is written.  The scales
 * are read for KV4 only. */
medusa_status medusa_kv_append(const medusa_cache* cache, const medusa_kv* kv,
                               const medusa_kv_rows* rows, const medusa_rope* rope, float k_scale,
                               float v_scale, void* stream);
/* Places that receive cached rows: item j of sequence b is slot first[b] + j (first NULL: j),
 * b and j from start or per_seq / count as in medusa_kv_rows.  Element strides as there. */
typedef struct {
  void* k;
  void* v;
  int dtype;                            /* MEDUSA_F32 or MEDUSA_BF16 */
  long long k_row, k_head, v_row, v_head;
  int rows;
  const int32_t* start;
  int per_seq;
  const int32_t* count;
  const int32_t* first;                 /* device [B] or NULL */
} medusa_kv_places;
/* Reads slots back (kv->k, v, page_table, len): what the cache holds, rounded once to dtype.
 * Only slots in [0, len[b]) are read (a len outside 0..capacity is taken as the nearer end, here and in
 * medusa_kv4_attention, without a flag); places of other slots are left as they were and set
 * MEDUSA_FLAG_KV_CAPACITY. */
medusa_status medusa_kv_read(const medusa_cache* cache, const medusa_kv* kv,
                             const medusa_kv_places* places, float k_scale, float v_scale,
                             void* stream);
/* Attention over a 4-bit cache: row n of sequence b, query head h attends to the slots
 * [0, len[b]) of key/value head h / (Hq/Hkv) and, where tree_k is given, to the call's own
 * rows j that n sees: bit j of mask row n (medusa_tree_build's mask), or j <= n without a mask.
 *   o = sum_j p_j v_j,  p = softmax(scale q . k_j)
 * One row (n1 = 1) is plain decoding: tree_k, tree_v are that token's keys/values, or NULL when
 * it has been appended already.  A row that sees nothing gives zeros, one that sees a NaN gives
 * NaN.  Slots from len[b] on and rows that are not seen may hold anything.  Calls that may run at
 * the same time need workspaces of their own.
 *   q: [B * n1] rows of Hq heads, element strides q_row, q_head; o: as q, strides o_row, o_head
 *   tree_k, tree_v: [B][n1][Hkv][dh]; q, o, tree_k, tree_v all of dtype (MEDUSA_F32 or
 *   MEDUSA_BF16), 16-byte aligned with strides of whole 16 bytes
 * Scores, softmax statistics and sums are 32 bits wide; scores beyond 2^107 in size may give any
 * result of that row's head.  With MEDUSA_F32 the products keep
 * 22 bits of queries and probabilities, with MEDUSA_BF16 the queries are exact (elements below
 * 2^-17 of a row's largest to 2^-25 of it) and the probabilities keep 11 bits. */
typedef struct {
  const void* q;
  void* o;
  int dtype;
  int n1;                               /* 1..max_nodes */
  long long q_row, q_head, o_row, o_head;
  const void* tree_k;
  const void* tree_v;
  const uint32_t* mask;                 /* device [n1][8] or NULL */
  float scale;                          /* 0: 1/sqrt(dh); at most 1e38 */
  float k_scale, v_scale;
} medusa_kv4_query;
medusa_status medusa_kv4_attention(const medusa_cache* cache, const medusa_kv* kv,
                                   const medusa_kv4_query* query, void* workspace,
                                   size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MEDUSA_H_ */
