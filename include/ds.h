/*
 * ds.h -- C ABI of the GB300 (sm_103a) tree-verify library.
 *
 * The library implements the target-model verify step of long-context
 * speculative decoding with a draft token tree:
 *
 *   ds_verify_attn        split-KV attention of every tree node over a paged
 *                         bf16 KV cache plus causal attention over the node's
 *                         own ancestors, emitting per-chunk attention mass
 *                         ("salience") in the same pass;
 *   ds_chunk_topk_gather  top-k chunks by salience plus a recent window,
 *                         gathered into a compact contiguous cache;
 *   ds_accept             the accepted path: greedy accept-if-equal or exact
 *                         tree rejection sampling with supplied uniforms
 *                         (ds_accept_static: the same over a scratch the
 *                         library owns, for callers that cannot allocate);
 *   ds_kv_commit          the accepted path's tree K/V moved behind the root
 *                         in every layer, and the new context lengths;
 *   ds_compact_append     newly committed tokens appended to the compact
 *                         cache between retrievals.
 *
 * and, for targets that keep their cache in 4 bits:
 *
 *   ds_qk_norm_rope       RMS norm of every query and key head and the position
 *                         rotation, in one pass over the projection's rows;
 *   ds_kv4_write          K/V rows quantised into the paged 4-bit cache (a
 *                         prompt, a tree, or the accepted path of a tree);
 *   ds_kv4_read           rows of the 4-bit cache read back as bf16;
 *   ds_kv4_verify_attn    ds_verify_attn over the 4-bit cache; a tree of one
 *                         node is plain decoding;
 *
 * and, for the draft model that decodes over the compact cache (or over a
 * paged one of its own):
 *
 *   ds_rope_frequencies   the rotation's frequencies, scaled for long contexts
 *                         (host only);
 *   ds_rope_append        queries and keys rotated, keys and values written
 *                         behind the cache's last slots (or the rotation alone,
 *                         or its inverse);
 *   ds_decode_attn        attention of one new token per sequence, every key's
 *                         weight added to its running sum;
 *   ds_cache_evict        a cache over its budget keeps its first and recent
 *                         tokens and the heaviest of the others.
 *
 * Conventions (all entry points):
 *   - Every pointer named in an args struct is a DEVICE pointer unless its
 *     comment says otherwise.  The caller owns every buffer, including the
 *     workspace; the library never allocates device memory.
 *   - Work is enqueued asynchronously on the caller's stream (`stream` is a
 *     cudaStream_t passed as void*; NULL is the legacy default stream).
 *   - Arguments are validated on the host before any work is enqueued.  A
 *     refused call returns DS_ERR_INVALID_ARG or DS_ERR_UNSUPPORTED and
 *     enqueues nothing; ds_last_error() then names the argument.
 *   - Values that live in device memory (lengths, parents, page ids, tokens)
 *     are checked by the kernels themselves.  A bad value never causes an
 *     out-of-bounds access: the affected sequence is skipped or the access
 *     is replaced by zeros, and a sticky bit is set in the workspace's
 *     status word (see ds_device_status).
 *   - bf16 means IEEE-754 binary32 truncated to its upper 16 bits (round to
 *     nearest even when produced), stored as uint16.
 */
#ifndef DS_VERIFY_H_
#define DS_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DS_ABI_VERSION 2
/* Largest draft tree per sequence: one 64-bit ancestor mask per node. */
#define DS_MAX_TREE_NODES 64

typedef enum {
  DS_OK = 0,
  DS_ERR_INVALID_ARG = 1,  /* a NULL pointer, negative size, bad enum, ...  */
  DS_ERR_UNSUPPORTED = 2,  /* a valid value the library does not support    */
  DS_ERR_CUDA = 3,         /* a CUDA runtime call or kernel launch failed   */
  DS_ERR_TIMEOUT = 4,      /* reserved: a bounded device-side wait gave up  */
  DS_ERR_WORKSPACE = 5     /* workspace missing, misaligned or too small    */
} ds_status;

/* Paged cache layouts.  NHD: [num_pages, page_size, num_kv_heads, head_dim];
 * HND: [num_pages, num_kv_heads, page_size, head_dim].  Both bf16, head_dim
 * contiguous.  Slot t of sequence b lives in page page_table[b][t/page_size]
 * at offset t % page_size. */
typedef enum { DS_KV_NHD = 0, DS_KV_HND = 1 } ds_kv_layout;

typedef enum { DS_OUT_BF16 = 0, DS_OUT_F32 = 1 } ds_out_dtype;

typedef enum { DS_ACCEPT_GREEDY = 0, DS_ACCEPT_REJECT = 1 } ds_accept_mode;

/* Sticky device-side status bits (ds_device_status). */
#define DS_DEV_BAD_LENGTH   0x1u  /* ctx_len < 0, or L+T beyond max_pages*page_size,
                                     or ceil(L/chunk) beyond max_chunks          */
#define DS_DEV_BAD_TREE     0x2u  /* tree size outside [0, 64], offsets not
                                     monotone, or a parent not an earlier node   */
#define DS_DEV_BAD_PAGE     0x4u  /* a page id outside [0, num_pages)            */
#define DS_DEV_BAD_TOKEN    0x8u  /* a draft token outside [0, vocab)            */
#define DS_DEV_TIMEOUT      0x10u /* a bounded wait inside a kernel gave up      */
#define DS_DEV_BAD_VALUE    0x20u /* a NaN or an infinity given to ds_kv4_write, a
                                     NaN among the weights of ds_cache_evict     */

/* Name of the last failure on the calling thread ("" if none).  The string is
 * owned by the library and valid until the next call on this thread. */
const char* ds_last_error(void);

/* Library ABI version (DS_ABI_VERSION of the build). */
int32_t ds_abi_version(void);

/* sizeof() of each args struct as compiled into the library: 0 verify,
 * 1 gather, 2 accept, 3 commit, 4 append, 5 norm_rope, 6 kv4_rows, 8 kv4_attn,
 * 9 rope_scaling, 10 rope, 11 decode, 12 evict; -1 for anything else (7 is not assigned).  Bindings compare these with their own struct layouts
 * before the first call. */
int64_t ds_struct_size(int32_t which);

/* Zero the whole workspace: the status word (bytes 0..255 of any workspace)
 * and the attention calls' split counters behind it (which every completed
 * call leaves at zero).  Call once after allocating a workspace, whenever the
 * sticky bits should be cleared, after a call that set DS_DEV_TIMEOUT (an
 * aborted call can leave counters behind), and before calls of another batch
 * size, of other head counts or of the other cache's attention on the same
 * workspace: the counters' number goes by these.  Everything else (nodes,
 * lengths, chunks, num_sms) may change from call to call.  Enqueued on
 * `stream`. */
ds_status ds_workspace_init(void* workspace, size_t workspace_bytes,
                            void* stream);

/* Copy the workspace's sticky status bits to *flags (host).  Synchronises
 * `stream` first.  0 means every device-side value checked so far was valid. */
ds_status ds_device_status(const void* workspace, uint32_t* flags,
                           void* stream);

/* ------------------------------------------------------------------------ *
 * Tree-verify attention with fused chunk salience.
 *
 * Defines (vllm-diffspec README, "What DiffSpec Does" items 2 and 5 and
 * "Architecture": chunks scored directly from paged target KV without
 * materialising the attention matrix; CGCL-codes/DiffSpec README,
 * "Features": salience-aware chunk encoding; adaptive-specdec README,
 * "Layout": the chain row mask s <= lengths[b] + j):
 *
 *   For sequence b with committed context length L = ctx_lens[b] and tree
 *   nodes n = tree_offsets[b] .. tree_offsets[b+1]-1 (local index j = n -
 *   tree_offsets[b], T = tree size <= 64, parents[n] local, -1 for j = 0),
 *   the tree's own keys and values sit in the paged cache at slots L + j.
 *   Query row (node j, query head h) attends, under kv head h / (Hq/Hkv),
 *   to every context slot t < L and to tree slot L + i iff i is j or an
 *   ancestor of j:
 *       s_t = scale * <q[n, h, :], k_t>,  p = softmax(s),
 *       out[n, h, :] = sum_t p_t v_t.
 *   chunk_scores[b, c] (= or +=, see accumulate_scores) is the attention
 *   mass that context chunk c = [c*C, min((c+1)*C, L)) receives, summed over
 *   all query heads and tree nodes of b, each row normalised by its full
 *   softmax denominator (context plus ancestors).  Only c < ceil(L/C) is
 *   written; other entries of the row are left untouched.
 *
 * Constraints refused with DS_ERR_UNSUPPORTED (by name):
 *   head_dim not 64 or 128; page_size not 16, 32, 64 or 128; chunk_size not
 *   a multiple of page_size or above 128 or not a power of two;
 *   num_q_heads not a multiple of num_kv_heads, or the group size
 *   num_q_heads / num_kv_heads not a power of two up to 16.
 * Alignment: q, caches, out and the workspace 16-byte aligned.
 * ------------------------------------------------------------------------ */
typedef struct ds_verify_args {
  const void*    q;             /* [n_nodes, num_q_heads, head_dim] bf16       */
  const void*    k_cache;       /* paged bf16, layout kv_layout                */
  const void*    v_cache;       /* paged bf16, same layout and page pool       */
  const int32_t* page_table;    /* [batch, max_pages] page ids                 */
  const int32_t* ctx_lens;      /* [batch] committed context length L_b >= 0   */
  const int32_t* tree_offsets;  /* [batch + 1], tree_offsets[0] = 0, last =
                                   n_nodes, nondecreasing                      */
  const int32_t* parents;       /* [n_nodes] local parent, -1 at local 0       */
  int32_t batch;                /* B >= 1                                      */
  int32_t n_nodes;              /* total tree nodes over the batch             */
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64 or 128                                   */
  int32_t page_size;
  int32_t num_pages;            /* pages in the pool (bounds page ids)         */
  int32_t max_pages;            /* row length of page_table                    */
  int32_t kv_layout;            /* ds_kv_layout                                */
  int32_t chunk_size;           /* C                                           */
  float   scale;                /* softmax scale; 0 selects 1/sqrt(head_dim)   */
  void*   out;                  /* [n_nodes, num_q_heads, head_dim]            */
  int32_t out_dtype;            /* ds_out_dtype                                */
  float*  chunk_scores;         /* [batch, max_chunks] fp32                    */
  int32_t max_chunks;           /* row length of chunk_scores                  */
  int32_t accumulate_scores;    /* 0: overwrite, 1: add (sum over layers).
                                   With 1 the call is a later layer of the
                                   step that began with 0: ctx_lens and
                                   tree_offsets must hold the same values and
                                   must not be written by the kernel issued
                                   right before this call on `stream` (they
                                   are read while that kernel may still run) */
  int32_t num_sms;              /* CTAs to plan for; 0 = the device's SM count */
  void*   workspace;            /* scratch, >= ds_verify_attn_workspace_size   */
  size_t  workspace_bytes;
  void*   prof_event_start;     /* optional cudaEvent_t (host handle) recorded
                                   on `stream` right before the split-pass
                                   kernel; NULL: not recorded                  */
  void*   prof_event_stop;      /* optional cudaEvent_t recorded right after it */
} ds_verify_args;

/* Fill *args with zeros/NULLs, kv_layout NHD, out_dtype BF16, scale 0. */
void ds_verify_args_default(ds_verify_args* args);

/* Bytes of workspace ds_verify_attn needs for these sizes (host only; reads
 * no pointer).  Depends on batch, n_nodes, head counts, head_dim, page_size,
 * max_pages, chunk_size, max_chunks and num_sms. */
ds_status ds_verify_attn_workspace_size(const ds_verify_args* args,
                                        size_t* bytes);

/* Enqueue the verify step.  Output `out` and `chunk_scores` are complete
 * when the work on `stream` completes.  The workspace must not be shared by
 * calls that may overlap on the GPU.  Its two kernels are launched as
 * programmatic dependents of the preceding work on `stream` (each waits for
 * that work to complete before it reads or writes memory, so ordering is
 * that of the stream; only launch latency overlaps); an event recorded
 * between two calls (for example `prof_event_*`) simply ends that overlap. */
ds_status ds_verify_attn(const ds_verify_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Top-k chunk selection plus recent window, gathered into a compact cache.
 *
 * Defines (vllm-diffspec README, "What DiffSpec Does", last paragraph:
 * selected chunks combined with a rolling recent window and rebuilt as a
 * compact cache; CGCL-codes/DiffSpec README, "Features": physically
 * contiguous chunk staging):
 *
 *   ws = max(0, L - window).  Candidates are the chunks wholly before the
 *   window, c with (c+1)*C <= ws.  The min(top_k, #candidates) candidates
 *   with the largest scores[b, c] (ties: lower c) are selected and listed in
 *   ascending order in out_chunk_ids[b, :] (-1 padded).  The working set is
 *   the selected chunks' tokens in ascending order followed by tokens
 *   [ws, L).  Token i of the working set, at absolute position t, is copied
 *   byte for byte from the paged source cache into out_k/out_v[b, i, :, :]
 *   and out_positions[b, i] = t; out_len[b] = working-set size.
 *   out_positions[b, i] = -1 for i >= out_len[b]; out_k/out_v rows beyond
 *   out_len[b] are left untouched.
 *
 *   With rope_base > 0 the source K is pre-RoPE and the compact cache is
 *   rebuilt with local positions (vllm-diffspec README, "Architecture":
 *   dual-view draft cache, canonical pre-RoPE KV at absolute positions and a
 *   compact cache with local draft RoPE positions): row i of out_k is the
 *   source row rotated to position i, pair (j, j + D/2) by the angle
 *   i * rope_base^(-2j/D), j < D/2, rounded to bf16.  The angle is reduced
 *   modulo one turn exactly (64-bit fixed point), its sine and cosine taken
 *   in float32 and the pair rotated in float32, so a value can differ from
 *   the exactly rounded result by one bf16 unit.  V is
 *   always copied byte for byte; rope_base = 0 copies K byte for byte too.
 *
 * Constraints: chunk_size a multiple of page_size; head_dim 64 or 128;
 * capacity >= top_k * chunk_size + window.
 * ------------------------------------------------------------------------ */
typedef struct ds_gather_args {
  const float*   scores;        /* [batch, max_chunks] fp32                    */
  int32_t        max_chunks;
  const int32_t* ctx_lens;      /* [batch]                                     */
  const void*    src_k;         /* paged bf16 source cache (kv_layout)         */
  const void*    src_v;
  const int32_t* page_table;    /* [batch, max_pages]                          */
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;
  int32_t chunk_size;
  int32_t top_k;                /* >= 0                                        */
  int32_t window;               /* >= 0                                        */
  int32_t capacity;             /* rows per sequence in out_k / out_v          */
  void*    out_k;               /* [batch, capacity, num_kv_heads, head_dim]   */
  void*    out_v;
  int32_t* out_positions;       /* [batch, capacity]                           */
  int32_t* out_len;             /* [batch]                                     */
  int32_t* out_chunk_ids;       /* [batch, top_k]                              */
  void*   workspace;            /* scratch, >= ds_chunk_topk_gather_workspace_size */
  size_t  workspace_bytes;
  float   rope_base;            /* 0: no rotation; > 0: RoPE base (theta)      */
} ds_gather_args;

void ds_gather_args_default(ds_gather_args* args);
ds_status ds_chunk_topk_gather_workspace_size(const ds_gather_args* args,
                                              size_t* bytes);
ds_status ds_chunk_topk_gather(const ds_gather_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Tree acceptance.
 *
 * Greedy (vllm.cpp docs "Speculative decoding", MTP: accept-if-equal):
 *   from the root (local node 0, whose draft token is ignored) repeatedly
 *   move to the first child, in increasing node index, whose draft token
 *   equals argmax_x target_logits[node, x] (lowest x on ties); stop when no
 *   child does.  bonus = that argmax at the stop node.
 * Rejection (adaptive-specdec README, "Correctness first" and "The
 *   controller"; children of a node are taken to be i.i.d. draws from its
 *   draft distribution):
 *   at node i, p = softmax(target[i]), q = softmax(draft[i]); for each
 *   child c in increasing node index with x = draft_tokens[c]: accept iff
 *   uniforms[c][0] * q(x) < p(x); on rejection p <- max(0, p - q) /
 *   sum(max(0, p - q)) (p kept when that sum is 0).  An accepted child
 *   becomes the current node.  With no child accepted, the bonus token is
 *   the smallest x with sum_{y <= x} p(y) > uniforms[i][1] * sum(p).  A
 *   draft token outside [0, vocab) at a non-root node sets DS_DEV_BAD_TOKEN
 *   and that node is never accepted.
 *
 * Outputs: out_path[b, 0..n-1] = accepted local node ids in order (-1
 * padded to DS_MAX_TREE_NODES), out_n_accepted[b] = n, out_bonus[b].  A
 * sequence with an empty tree gets n = 0 and bonus -1.
 * ------------------------------------------------------------------------ */
typedef struct ds_accept_args {
  int32_t        mode;          /* ds_accept_mode                              */
  const float*   target_logits; /* [n_nodes, vocab] fp32                       */
  const float*   draft_logits;  /* [n_nodes, vocab] fp32; NULL when greedy     */
  const int32_t* draft_tokens;  /* [n_nodes]                                   */
  const int32_t* parents;       /* [n_nodes] local parent, -1 at local 0       */
  const int32_t* tree_offsets;  /* [batch + 1]                                 */
  const float*   uniforms;      /* [n_nodes, 2] in [0, 1); NULL when greedy    */
  int32_t batch;
  int32_t n_nodes;
  int32_t vocab;
  int32_t* out_path;            /* [batch, DS_MAX_TREE_NODES]                  */
  int32_t* out_n_accepted;      /* [batch]                                     */
  int32_t* out_bonus;           /* [batch]                                     */
  void*   workspace;            /* scratch, >= ds_accept_workspace_size        */
  size_t  workspace_bytes;
} ds_accept_args;

void ds_accept_args_default(ds_accept_args* args);
ds_status ds_accept_workspace_size(const ds_accept_args* args, size_t* bytes);
ds_status ds_accept(const ds_accept_args* args, void* stream);

/* Tree acceptance without a caller-supplied workspace.  The method itself
 * has no counterpart to this entry: it is ds_accept for callers that cannot
 * hand out device memory where they call it (a plugin or host callback
 * whose framework owns every allocation and gives it no allocator, or a
 * serving loop that forbids allocation once warm).
 *
 * Same arguments, kernels and results as ds_accept, except that
 * args->workspace must be NULL and args->workspace_bytes 0: the scratch
 * (a status word and one 96-byte record per tree node) is a fixed array in
 * device global memory inside the library, DS_ACCEPT_STATIC_MAX_NODES
 * records long (384 KiB per device).  Nothing is allocated, on the
 * device or through any library, by this call.
 *
 * Refused with DS_ERR_UNSUPPORTED: args->n_nodes > DS_ACCEPT_STATIC_MAX_NODES
 * (use ds_accept).  Refused with DS_ERR_INVALID_ARG: a non-NULL workspace.
 *
 * Every call looks up the array's address in the current context
 * (cudaGetSymbolAddress, which allocates nothing), so a context torn down
 * and created again (cudaDeviceReset) is followed correctly; make one call
 * before capturing `stream` into a graph, so that the module is loaded
 * outside the capture.  Each call then enqueues, on `stream`, a zeroing of
 * the status word (the one part of the scratch that must start at zero;
 * the node records are written before they are read) and the acceptance
 * kernels.
 *
 * flags_out: NULL to return as soon as the work is enqueued; otherwise the
 * call synchronises `stream` and stores this call's device status bits
 * (DS_DEV_BAD_TREE, DS_DEV_BAD_TOKEN; 0 = inputs valid) at *flags_out.
 *
 * One scratch per device: two calls whose work may overlap on the device
 * (different streams, or different host threads, without ordering between
 * them) race on it and give undefined results.  Serialise them. */
#define DS_ACCEPT_STATIC_MAX_NODES 4096
ds_status ds_accept_static(const ds_accept_args* args, uint32_t* flags_out,
                           void* stream);

/* ------------------------------------------------------------------------ *
 * Compact-cache append between retrievals (vllm-diffspec README, "What
 * DiffSpec Does" item 4: KV reuse and locality across decoding steps, and
 * "Configuration": diffspec_retrieval_interval, verifier cycles between
 * retrievals).
 *
 * The compact cache built by ds_chunk_topk_gather is kept; for every
 * sequence b the tokens committed since, t in [from_lens[b], to_lens[b]),
 * are copied from the paged source cache behind its last row: row
 * out_len[b] + (t - from_lens[b]) gets token t, out_positions of that row is
 * t, K is rotated to that row's local position when rope_base > 0 (as in
 * ds_chunk_topk_gather), and out_len[b] grows by to - from.  If the rows do
 * not fit in capacity, or from > to, or to is beyond max_pages * page_size,
 * nothing is appended for b and DS_DEV_BAD_LENGTH is set; a page id outside
 * [0, num_pages) sets DS_DEV_BAD_PAGE and that row is written as zeros.
 * Refused on the host: head_dim not 64 or 128, capacity < 0, rope_base < 0.
 * ------------------------------------------------------------------------ */
typedef struct ds_append_args {
  const void*    src_k;         /* paged bf16 source cache (pre-RoPE K)       */
  const void*    src_v;
  const int32_t* page_table;    /* [batch, max_pages]                         */
  const int32_t* from_lens;     /* [batch]                                    */
  const int32_t* to_lens;       /* [batch]                                    */
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;
  int32_t capacity;             /* rows per sequence of the compact cache     */
  void*    out_k;               /* [batch, capacity, num_kv_heads, head_dim]  */
  void*    out_v;
  int32_t* out_positions;       /* [batch, capacity]                          */
  int32_t* out_len;             /* [batch] rows present; updated in place     */
  float    rope_base;           /* 0: K copied byte for byte                  */
  void*   workspace;            /* >= 256 bytes: the status word              */
  size_t  workspace_bytes;
} ds_append_args;

void ds_append_args_default(ds_append_args* args);
ds_status ds_compact_append(const ds_append_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Post-accept KV commit (adaptive-specdec README, "Layout": one cache buffer
 * per layer, a per-sequence lengths vector, writes scattered to each row's
 * own offset, rollback by length).
 *
 * For every sequence b with a tree (T = tree_offsets[b+1] - tree_offsets[b]
 * >= 1) and L = ctx_lens[b]: the root's K/V (node 0) already sits at slot L;
 * the accepted nodes c_1 < ... < c_n (path[b, 0..n-1], n = n_accepted[b], as
 * ds_accept writes them) are copied, in every layer and kv head, K and V,
 * from slot L + c_i to slot L + i, and new_ctx_lens[b] = L + 1 + n.  Slots
 * past the new length keep stale data that the length excludes.  A sequence
 * without a tree gets new_ctx_lens[b] = L.
 *
 * Device-side checks (status bits in the workspace, see ds_device_status):
 * a path that is not strictly increasing inside (0, T) or n outside
 * [0, T-1] sets DS_DEV_BAD_TREE and commits the root only (L + 1); a page id
 * outside [0, num_pages) sets DS_DEV_BAD_PAGE and that slot is skipped;
 * L + T beyond max_pages * page_size sets DS_DEV_BAD_LENGTH and the sequence
 * keeps L.  Refused on the host: num_layers outside 1..DS_MAX_COMMIT_LAYERS,
 * head_dim not 64 or 128, page_size not 16/32/64/128, new_ctx_lens == ctx_lens.
 * Caches as in ds_verify_attn (same layout for all layers), 16-byte aligned.
 * ------------------------------------------------------------------------ */
#define DS_MAX_COMMIT_LAYERS 128

typedef struct ds_commit_args {
  void* const*   k_caches;      /* host array [num_layers] of device pointers   */
  void* const*   v_caches;      /* host array [num_layers] of device pointers   */
  int32_t        num_layers;
  const int32_t* page_table;    /* [batch, max_pages]                           */
  const int32_t* ctx_lens;      /* [batch]                                      */
  const int32_t* tree_offsets;  /* [batch + 1]                                  */
  const int32_t* path;          /* [batch, DS_MAX_TREE_NODES] from ds_accept    */
  const int32_t* n_accepted;    /* [batch]                                      */
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;            /* ds_kv_layout                                 */
  int32_t* new_ctx_lens;        /* [batch] out; must not alias ctx_lens         */
  void*   workspace;            /* >= 256 bytes: the status word                */
  size_t  workspace_bytes;
} ds_commit_args;

void ds_commit_args_default(ds_commit_args* args);
ds_status ds_kv_commit(const ds_commit_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Norm of every query and key head with the position rotation, in one pass.
 *
 * For every row n (a token or a tree node) and every query and key head x of
 * head_dim values:
 *   y = x * w / sqrt(mean(x^2) + eps)      (w = q_weight / k_weight; y = x
 *                                           when that weight is NULL)
 *   out[j]       = y[j] cos(a_j) - y[j + D/2] sin(a_j)
 *   out[j + D/2] = y[j] sin(a_j) + y[j + D/2] cos(a_j),   j < D/2,
 * a_j = positions[n] * rope_base^(-2j/D), or positions[n] * inv_freq[j] when
 * inv_freq is given (for scaled rotations).  Both 0 / NULL: no rotation.
 * The sum of squares, the norm and the rotation are float32, the angle is
 * reduced modulo one turn in 64-bit fixed point (as in ds_chunk_topk_gather),
 * and each value is rounded to bf16 once.
 *
 * Rows may be slices of a wider buffer (the fused projection's output): the
 * row strides are in elements, heads of a row are head_dim apart.  q_out may
 * be q itself and k_out k itself, with the same stride; otherwise outputs
 * must not overlap inputs.  num_q_heads or num_kv_heads may be 0.  A negative
 * position sets DS_DEV_BAD_LENGTH and that row is not written.
 *
 * Refused: head_dim not 64 or 128; pointers not 16-byte aligned or strides
 * not a multiple of 8 or shorter than a row; eps negative or not finite.
 * ------------------------------------------------------------------------ */
typedef struct ds_norm_rope_args {
  const void*    q;             /* n_rows rows of num_q_heads x head_dim bf16    */
  const void*    k;             /* n_rows rows of num_kv_heads x head_dim bf16   */
  int64_t        q_row_stride;  /* elements from a row to the next               */
  int64_t        k_row_stride;
  const void*    q_weight;      /* [head_dim] bf16; NULL: queries not normed     */
  const void*    k_weight;      /* [head_dim] bf16; NULL: keys not normed        */
  const int32_t* positions;     /* [n_rows] absolute positions >= 0              */
  int32_t n_rows;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64 or 128                                     */
  float   eps;
  float   rope_base;            /* 0: see inv_freq                               */
  const double*  inv_freq;      /* HOST array [head_dim / 2] of radians per
                                   position, or NULL; needs rope_base 0          */
  void*   q_out;
  void*   k_out;
  int64_t q_out_row_stride;
  int64_t k_out_row_stride;
  void*   workspace;            /* >= 256 bytes: the status word                 */
  size_t  workspace_bytes;
} ds_norm_rope_args;

void ds_norm_rope_args_default(ds_norm_rope_args* args);
ds_status ds_qk_norm_rope(const ds_norm_rope_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * The 4-bit paged cache.
 *
 * A value is  code * scale * 2^exp: an e2m1 code (magnitudes 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6), an e4m3 scale shared by 16 consecutive channels of one
 * token's head, and one exponent per tensor (k_exp, v_exp; both are host
 * integers that every call on the cache must repeat).  4.5 bits per value;
 * code * scale has at most six significant bits, so bf16 holds it exactly.
 *
 * K and V are pools [num_pages, num_kv_heads, block] of bytes, block =
 * DS_KV4_BLOCK_BYTES(page_size, head_dim): the codes [page_size][head_dim/2]
 * (channel 2i in the low nibble of byte i, 2i + 1 in the high), then the
 * scales [page_size][head_dim/16].  Slot t of sequence b lives in page
 * page_table[b][t / page_size] at offset t % page_size, as in the bf16 cache.
 *
 * Quantising x (16 channels): y = x 2^-exp; scale = max|y| / 6 rounded to the
 * nearest e4m3 (ties to even, at most 448); code = y / scale rounded to the
 * nearest e2m1 (ties to even, at most 6); scale 0 gives codes 0.  All of it
 * is exact but for these two roundings.  A NaN is stored as 0 and an
 * infinity as the largest value; both set DS_DEV_BAD_VALUE.  Readers take
 * the two e4m3 patterns that are no number (0x7f, 0xff) as 448, so no byte
 * of a cache, written or not, ever reads as NaN or infinity.
 * ------------------------------------------------------------------------ */
#define DS_KV4_BLOCK_BYTES(page_size, head_dim) ((page_size) * (head_dim) * 9 / 16)

/* Rows and slots: row row_offsets[b] + i of sequence b belongs to slot
 * from_lens[b] + i.
 *
 * ds_kv4_write quantises the rows into their slots.  With `path` (and
 * n_accepted, as ds_accept writes them) it commits a tree instead: the rows
 * are the tree's (at most DS_MAX_TREE_NODES per sequence), and row
 * row_offsets[b] + path[b, i] goes to slot from_lens[b] + 1 + i, i <
 * n_accepted[b]; the root stays where the tree was written.  new_lens[b],
 * when given, is the length that follows: from_lens[b] + rows of b, or
 * from_lens[b] + 1 + n_accepted[b] with a path (from_lens[b] for an empty
 * tree).  A path that is not strictly increasing inside (0, rows of b) sets
 * DS_DEV_BAD_TREE and commits the root only.
 *
 * ds_kv4_read writes the rows from their slots, as bf16 (exactly; path,
 * n_accepted and new_lens must be NULL).
 *
 * Both: a length below 0, past max_pages * page_size or row offsets that
 * decrease or leave [0, n_rows] set DS_DEV_BAD_LENGTH and skip the sequence
 * (new_lens[b] is from_lens[b] then; with n_rows 0 and no new_lens there is
 * nothing to do and nothing is looked at);
 * a page id outside [0, num_pages) sets DS_DEV_BAD_PAGE, and that slot is
 * not written (its row reads as zeros).  Two rows must not share a slot.
 * Refused: head_dim not 64 or 128; page_size not 16, 32, 64 or 128;
 * exponents outside [-32, 32]; rows or caches not 16-byte aligned; strides
 * not a multiple of 8 or shorter than a row; new_lens == from_lens. */
typedef struct ds_kv4_rows_args {
  void*   k_rows;               /* n_rows rows of num_kv_heads x head_dim bf16
                                   (ds_kv4_write only reads them)                */
  void*   v_rows;
  int64_t k_row_stride;         /* elements from a row to the next               */
  int64_t v_row_stride;
  void*   k_cache;              /* 4-bit pools (ds_kv4_read only reads them)     */
  void*   v_cache;
  const int32_t* page_table;    /* [batch, max_pages]                            */
  const int32_t* from_lens;     /* [batch] slot of each sequence's first row     */
  const int32_t* row_offsets;   /* [batch + 1]                                   */
  const int32_t* path;          /* [batch, DS_MAX_TREE_NODES] or NULL            */
  const int32_t* n_accepted;    /* [batch]; NULL without a path                  */
  int32_t batch;
  int32_t n_rows;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t k_exp;
  int32_t v_exp;
  int32_t* new_lens;            /* [batch] out, or NULL                          */
  void*   workspace;            /* >= 256 bytes: the status word                 */
  size_t  workspace_bytes;
} ds_kv4_rows_args;

void ds_kv4_rows_args_default(ds_kv4_rows_args* args);
ds_status ds_kv4_write(const ds_kv4_rows_args* args, void* stream);
ds_status ds_kv4_read(const ds_kv4_rows_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Tree-verify attention over the 4-bit cache.
 *
 * ds_verify_attn (the same trees, masks, outputs, chunk salience, device-side
 * checks and dependent launches) over K and V in the 4-bit cache.  The tree's
 * own keys and values are in the cache too, at slots L + j (ds_kv4_write
 * puts them there).  A batch whose trees have one node each is a decoding
 * step.  Queries enter the product as float16: those beyond +-65504 are
 * clamped to it (a NaN stays one), and the bits of a bf16 query below 2^-24
 * are rounded off.  Weights enter the second product as float16 too; maxima,
 * sums and outputs in progress are float32, and outputs that splits exchange
 * float16 or float32.
 *
 * chunk_scores NULL: no salience (chunk_size, max_chunks and
 * accumulate_scores are then ignored).  A page id outside [0, num_pages)
 * sets DS_DEV_BAD_PAGE and its slots read as zeros.  Offsets that are not
 * monotone set DS_DEV_BAD_TREE; when they describe more nodes than n_nodes, the
 * call may write nothing.  The workspace's size does not depend on n_nodes.
 * Refused by name: as ds_verify_attn, and exponents outside [-32, 32],
 * scale * 2^k_exp beyond float32 and max_pages * page_size above 2^30. */
typedef struct ds_kv4_attn_args {
  const void*    q;             /* [n_nodes, num_q_heads, head_dim] bf16         */
  const void*    k_cache;       /* 4-bit pools                                   */
  const void*    v_cache;
  const int32_t* page_table;    /* [batch, max_pages]                            */
  const int32_t* ctx_lens;      /* [batch]                                       */
  const int32_t* tree_offsets;  /* [batch + 1]                                   */
  const int32_t* parents;       /* [n_nodes]                                     */
  int32_t batch;
  int32_t n_nodes;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t chunk_size;
  float   scale;                /* softmax scale; 0 selects 1/sqrt(head_dim)     */
  int32_t k_exp;
  int32_t v_exp;
  void*   out;                  /* [n_nodes, num_q_heads, head_dim]              */
  int32_t out_dtype;            /* ds_out_dtype                                  */
  float*  chunk_scores;         /* [batch, max_chunks] fp32, or NULL             */
  int32_t max_chunks;
  int32_t accumulate_scores;    /* as in ds_verify_args                          */
  int32_t num_sms;              /* CTAs to plan for; 0 = the device's SM count   */
  void*   workspace;            /* >= ds_kv4_verify_attn_workspace_size          */
  size_t  workspace_bytes;
} ds_kv4_attn_args;

void ds_kv4_attn_args_default(ds_kv4_attn_args* args);
ds_status ds_kv4_verify_attn_workspace_size(const ds_kv4_attn_args* args,
                                            size_t* bytes);
ds_status ds_kv4_verify_attn(const ds_kv4_attn_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * The draft's cache.
 *
 * The three calls below work on one layer's K/V cache of bf16 or f16 values,
 * in one of two forms:
 *   paged    (page_table given) as in ds_verify_attn: slot t of sequence b is
 *            at offset t % page_size of page page_table[b][t / page_size];
 *            page_size 16, 32, 64 or 128;
 *   compact  (page_table NULL) as ds_chunk_topk_gather writes it: sequence b's
 *            slots are page b, [batch, page_size, num_kv_heads, head_dim] (or
 *            heads before slots with DS_KV_HND), page_size any capacity >= 1,
 *            num_pages >= batch; max_pages is ignored.
 * A sequence has max_pages * page_size slots (page_size when compact), at
 * most 2^30.  Beside the cache a program may keep, per slot, the token's
 * position (int32) and the sum of the attention weight it has received (f32),
 * both [batch, slot_heads, slot_stride]: slot_heads 1 when all kv heads keep
 * the same tokens, num_kv_heads when each keeps its own; slot_stride at least
 * the slots of a sequence.  Slots need not be in order of position.
 *
 * Caches must be 16-byte aligned; head_dim 64 or 128.
 * ------------------------------------------------------------------------ */
typedef enum { DS_KV_BF16 = 0, DS_KV_F16 = 1 } ds_kv_dtype;

/* Which two values of a head's first rotary_dim = r are rotated together:
 * (j, j + r/2) or (2j, 2j + 1), j < r/2. */
typedef enum { DS_ROPE_HALF = 0, DS_ROPE_INTERLEAVED = 1 } ds_rope_layout;

/* Frequencies scaled for contexts longer than those of training.  Pair j has
 * th = base^(-2j/r) radians per position; o = original_len, f = factor, and
 * turns = o th / (2 pi), the pair's turns over the original length:
 *   NONE    th
 *   LINEAR  th / f
 *   BANDS   th (s + (1 - s) / f), s = (turns - low) / (high - low) clamped to
 *           [0, 1]: pairs of more than `high` turns as they are, those of
 *           fewer than `low` divided by f
 *   RAMP    th (1 - g + g / f), g = (j - lo) / (hi - lo) clamped to [0, 1],
 *           d(n) = r ln(o / (2 pi n)) / (2 ln base), lo = max(0, floor
 *           d(high)), hi = min(r - 1, ceil d(low)) (a denominator of zero or
 *           less counts as 0.001); magnitude 0.1 ln f + 1
 * The magnitude (1 but for RAMP) multiplies cosines and sines. */
typedef enum {
  DS_ROPE_SCALE_NONE = 0,
  DS_ROPE_SCALE_LINEAR = 1,
  DS_ROPE_SCALE_BANDS = 2,
  DS_ROPE_SCALE_RAMP = 3
} ds_rope_scale;

typedef struct ds_rope_scaling {
  int32_t kind;                 /* ds_rope_scale                                 */
  int32_t rotary_dim;           /* r: even, 2 to 128                             */
  double  base;                 /* > 1                                           */
  double  factor;               /* f >= 1 (all but NONE)                         */
  double  original_len;         /* o > 0 (BANDS, RAMP)                           */
  double  low;                  /* turns, 0 < low < high (BANDS, RAMP)           */
  double  high;
} ds_rope_scaling;

/* Zeros, kind NONE, factor 1. */
void ds_rope_scaling_default(ds_rope_scaling* scaling);

/* inv_freq[rotary_dim / 2] (HOST) in radians per position, for inv_freq of
 * ds_rope_append and ds_qk_norm_rope, and *magnitude (HOST).  Host only.
 * Refused: a value outside the ranges above, or not finite. */
ds_status ds_rope_frequencies(const ds_rope_scaling* scaling, double* inv_freq,
                              float* magnitude);

/* ------------------------------------------------------------------------ *
 * Rotation by position, and the new tokens' rows into the cache.
 *
 * For every row n (a token) and every query and key head x, with
 * a_j = positions[n] * inv_freq[j] (or * rope_base^(-2j/r)) and m = magnitude:
 *   (x_j, x_j') -> m (x_j cos a_j - x_j' sin a_j, x_j sin a_j + x_j' cos a_j)
 * for the r/2 pairs (j, j') of `layout`; the values from r on are copied.
 * With inverse = 1 the angles are -a_j: m times the transpose of the matrix
 * without it, so that dL/dx = the inverse rotation of dL/dy (with the same m).
 * Angles are reduced modulo one turn in 64-bit fixed point, sines, cosines and
 * products are float32, and each value is rounded once.
 *
 * k_cache NULL: the rotation alone, q into q_out and k into k_out; v and the
 * fields of the cache are ignored.
 *
 * With a cache, row row_offsets[b] + i of sequence b belongs to slot
 * from_lens[b] + i: the rotated key and the value go there (and the key into
 * k_out too when that is not NULL), slot_positions[b, :, slot] = positions[n]
 * and slot_weights[b, :, slot] = 0 when given, and new_lens[b] = from_lens[b]
 * + rows of b when given.  Rows that belong to no sequence, or to one that is
 * refused, are left out altogether, q_out included.  Two rows must not share
 * a slot.
 *
 * Rows may be slices of a wider buffer, as in ds_qk_norm_rope.  q_out may be q
 * and k_out may be k, with the same stride; outputs must not overlap inputs
 * otherwise.  num_q_heads 0 (no queries) or, without a cache, num_kv_heads 0
 * is allowed.
 *
 * Checked on the device: a negative position sets DS_DEV_BAD_LENGTH and that
 * row is left out (its slot keeps what it holds; new_lens counts it); a
 * from_lens below 0, rows beyond the sequence's slots, or row offsets that
 * decrease or leave [0, n_rows] set DS_DEV_BAD_LENGTH and leave the sequence
 * out (new_lens[b] is from_lens[b] then); a page id outside [0, num_pages)
 * sets DS_DEV_BAD_PAGE, and that slot's key and value are not written
 * (new_lens counts it).  Where offsets decrease or leave the rows,
 * other sequences' rows can be in doubt: one that a search of the offsets does
 * not find for each of its rows is left out too.  It finds every sequence of
 * which no earlier offset lies above its first row and no later one below its
 * end.  (A paged sequence of which no row has a page has nothing to write when
 * slot_positions and slot_weights are NULL: new_lens counts its rows then.)
 *
 * Refused: head_dim not 64 or 128; rotary_dim not a multiple of 16 up to
 * head_dim; pointers not 16-byte aligned or strides not a multiple of 8 or
 * shorter than a row; new_lens == from_lens; enums out of range; magnitude,
 * inv_freq or rope_base not finite, or neither or both of the last two given.
 * ------------------------------------------------------------------------ */
typedef struct ds_rope_args {
  const void*    q;             /* n_rows rows of num_q_heads x head_dim         */
  const void*    k;             /* n_rows rows of num_kv_heads x head_dim        */
  const void*    v;             /* the same; only with a cache                   */
  int64_t        q_row_stride;  /* elements from a row to the next               */
  int64_t        k_row_stride;
  int64_t        v_row_stride;
  const int32_t* positions;     /* [n_rows] >= 0                                 */
  int32_t n_rows;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64 or 128                                     */
  int32_t dtype;                /* ds_kv_dtype of rows, outputs and cache        */
  int32_t layout;               /* ds_rope_layout                                */
  int32_t rotary_dim;           /* r; 0 selects head_dim                         */
  int32_t inverse;              /* 0 or 1                                        */
  float   rope_base;            /* > 0, or 0 with inv_freq                       */
  float   magnitude;            /* m; default 1                                  */
  const double*  inv_freq;      /* HOST array [r / 2], or NULL with rope_base    */
  void*   q_out;
  void*   k_out;                /* NULL: none (with a cache)                     */
  int64_t q_out_row_stride;
  int64_t k_out_row_stride;
  void*   k_cache;              /* NULL: rotation alone                          */
  void*   v_cache;
  const int32_t* page_table;    /* [batch, max_pages]; NULL: compact             */
  const int32_t* from_lens;     /* [batch] slot of each sequence's first row     */
  const int32_t* row_offsets;   /* [batch + 1]                                   */
  int32_t batch;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;            /* ds_kv_layout                                  */
  int32_t slot_heads;           /* 1 or num_kv_heads; of the next two            */
  int64_t slot_stride;
  int32_t* slot_positions;      /* [batch, slot_heads, slot_stride] or NULL      */
  float*   slot_weights;        /* the same, or NULL                             */
  int32_t* new_lens;            /* [batch] out, or NULL                          */
  void*   workspace;            /* >= 256 bytes: the status word                 */
  size_t  workspace_bytes;
} ds_rope_args;

void ds_rope_args_default(ds_rope_args* args);
ds_status ds_rope_append(const ds_rope_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Attention of one new token per sequence.
 *
 * Sequence b has n = lens[b] slots (the new token's own among them, when it
 * was appended).  Query head h attends, under kv head h / (Hq/Hkv), to the
 * slots t < n, with window > 0 only to t >= n - window and to t < sinks:
 *   s_t = scale * <q[b, h, :], k_t>,  p = softmax(s),
 *   out[b, h, :] = sum_t p_t v_t,  lse[b, h] = ln sum_t exp(s_t).
 * A sequence without slots gets out 0 and lse -inf.
 *
 * With weights_out every slot t < n gets
 *   weights_out[b, w, t] = decay * weights_in[b, w, t] + sum of p_t
 * over the query heads of kv head w (slot_heads = num_kv_heads) or over all
 * query heads (slot_heads = 1); p_t is 0 for slots that are not attended to.
 * weights_in NULL counts as zeros; it may be weights_out.  Slots from n on
 * are left as they were.
 *
 * `window` and `sinks` count slots here, not positions.  Where slots are not in
 * order of position (a retrieved cache, or one that ds_cache_evict has cut) the
 * last slots are not the last tokens, and a window is no sliding window of them;
 * ds_cache_evict's `recent` and `sinks` go by position.
 *
 * Products are float32 sums of exact products; each weight enters the second
 * product as the sum of two values of the cache's type, which is exact to
 * 2^-16 of it (bf16; f16: 2^-22, or 2^-32 of the row's largest); maxima, sums,
 * and what splits exchange are float32.
 * What lies in slots that are not attended to (NaN included) has no effect.
 * An infinite value that is attended to makes its channel's output infinite,
 * however small its weight; NaN, both signs, or a logit of -inf beside it make
 * it NaN.  Outputs are divided by the sum of weights at the end: in bf16, |v|
 * times that sum over the largest weight must stay below 2^119.
 * No state is kept in the workspace from call to call.
 *
 * Checked on the device: a length below 0 or beyond the sequence's slots sets
 * DS_DEV_BAD_LENGTH and counts as 0; a page id outside [0, num_pages) sets
 * DS_DEV_BAD_PAGE and its slots read as zeros.  Pages of which no slot is
 * attended to are not looked up.
 * Refused: head_dim not 64 or 128; num_q_heads not a multiple of
 * num_kv_heads, or more than 16 query heads to a kv head; pointers not 16-byte
 * aligned; q_row_stride not a multiple of 8 or shorter than a row; window,
 * sinks, decay or scale negative or not finite; batch above 65,536.
 * ------------------------------------------------------------------------ */
typedef struct ds_decode_args {
  const void*    q;             /* [batch] rows of num_q_heads x head_dim        */
  int64_t        q_row_stride;  /* elements from a row to the next               */
  const void*    k_cache;
  const void*    v_cache;
  const int32_t* page_table;    /* [batch, max_pages]; NULL: compact             */
  const int32_t* lens;          /* [batch]                                       */
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64 or 128                                     */
  int32_t dtype;                /* ds_kv_dtype of q and the cache                */
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;            /* ds_kv_layout                                  */
  float   scale;                /* softmax scale; 0 selects 1/sqrt(head_dim)     */
  int32_t window;               /* 0: all slots                                  */
  int32_t sinks;
  void*   out;                  /* [batch, num_q_heads, head_dim]                */
  int32_t out_f32;              /* 0: out has dtype, 1: float32                  */
  float*  lse;                  /* [batch, num_q_heads], or NULL                 */
  const float* weights_in;      /* [batch, slot_heads, slot_stride], or NULL     */
  float*  weights_out;          /* the same, or NULL: no weights are formed      */
  float   decay;                /* default 1                                     */
  int32_t slot_heads;           /* 1 or num_kv_heads                             */
  int64_t slot_stride;
  int32_t num_sms;              /* CTAs to plan for; 0 = the device's SM count   */
  void*   workspace;            /* >= ds_decode_attn_workspace_size              */
  size_t  workspace_bytes;
} ds_decode_args;

void ds_decode_args_default(ds_decode_args* args);
/* Depends on the sizes, on num_sms and on whether weights_out is given (then
 * it holds a float32 per query head and slot that a sequence has room for,
 * whatever the lengths: 604 MB for 256 sequences of 32 heads and 18,432 slots). */
ds_status ds_decode_attn_workspace_size(const ds_decode_args* args, size_t* bytes);
ds_status ds_decode_attn(const ds_decode_args* args, void* stream);

/* ------------------------------------------------------------------------ *
 * Eviction by accumulated attention weight, in place.
 *
 * A sequence of n = lens[b] slots is cut when n > max(budget, trigger), to
 * `budget` slots, per slot head w (all kv heads together when slot_heads is
 * 1): slots whose position is below `sinks`, or at least next_positions[b] -
 * recent, come first, then those of the larger weight, of equal ones (-0 is
 * 0) the lower slot; a NaN counts as lighter than any weight and sets
 * DS_DEV_BAD_VALUE.  The first `budget` in this order are kept.  Kept slots
 * below `budget` stay where they are; the kept slots from `budget` on move, in
 * ascending order, into the slots below `budget` that are given up, ascending:
 * K, V, position and weight.  new_lens[b] = budget.  Slots from `budget` on
 * keep what they hold.  A sequence that is not cut keeps its n slots, and
 * new_lens[b] = n.
 *
 * weights_out and positions_out, when given, receive the slots below new_lens
 * and leave the inputs as they were (they must not overlap them, or be the
 * inputs themselves, which is the same as NULL: in place).
 *
 * Rows move within a sequence's own pages: a page must belong to one sequence
 * only, or another that shares it (a common prefix) loses its tokens.  What was
 * given up is gone: tokens appended last can be taken back by a shorter length
 * only while nothing has been evicted since, and what they added to the other
 * slots' weights stays.
 *
 * Checked on the device: a length below 0 or beyond the sequence's slots sets
 * DS_DEV_BAD_LENGTH and the sequence is left alone (new_lens[b] = lens[b]); a
 * page id outside [0, num_pages) sets DS_DEV_BAD_PAGE, and that token's key and
 * value are not moved.  No state is kept in the workspace from call to call.
 * Refused: budget below 1; recent + sinks above it; trigger, recent or sinks
 * negative; new_lens == lens; sizes as in the calls above; batch *
 * slot_heads above 65,536.
 * ------------------------------------------------------------------------ */
typedef struct ds_evict_args {
  void*   k_cache;
  void*   v_cache;
  const int32_t* page_table;    /* [batch, max_pages]; NULL: compact             */
  const int32_t* lens;          /* [batch]                                       */
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64 or 128 (values of two bytes of any type)   */
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t kv_layout;            /* ds_kv_layout                                  */
  int32_t slot_heads;           /* 1 or num_kv_heads                             */
  int64_t slot_stride;
  float*   weights;             /* [batch, slot_heads, slot_stride]              */
  int32_t* positions;
  float*   weights_out;         /* the same, or NULL: in place                   */
  int32_t* positions_out;
  const int32_t* next_positions; /* [batch] position of the next token           */
  int32_t budget;
  int32_t trigger;              /* 0: budget                                     */
  int32_t recent;
  int32_t sinks;
  int32_t* new_lens;            /* [batch] out                                   */
  void*   workspace;            /* >= ds_cache_evict_workspace_size              */
  size_t  workspace_bytes;
} ds_evict_args;

void ds_evict_args_default(ds_evict_args* args);
ds_status ds_cache_evict_workspace_size(const ds_evict_args* args, size_t* bytes);
ds_status ds_cache_evict(const ds_evict_args* args, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* DS_VERIFY_H_ */
