/*
 * zha.h -- C ABI of the ZHA decode hot path on B200 (sm_100a): tree-summarised
 * KV-cache attention.
 *
 * Citations name a page by its title and a section on it:
 *   [ZHA: <section>]  page "ZHA는 KV 캐시를 트리로 요약해 어텐션 비용을 준(sub)이차로
 *                     낮춘다" (onedev.kr/papers/1556);
 *   [Attention: <section>]  page "Attention"
 *                     (zzong2006.github.io/machine_learning/nlp/attention-function).
 *
 * The method: every contiguous key chunk of C tokens gets, at each of R
 * reference queries q_r, a tangent plane t_r(q) = q.khat_r/sqrt(d) + bhat_r of
 * its log attention mass; level l >= 2 nodes merge C children the same way.
 * At decode time each query head is routed level by level with top-p over the
 * planes' maximum, and exact softmax attention runs over the gathered leaf
 * tokens, the sink (token 0) and the in-progress tail [ZHA: 무엇과 다른가,
 * 전제와 한계]. One tree per KV head serves its GQA query heads.
 *
 * Conventions for every call:
 *  - All pointers named d_* are DEVICE pointers owned by the caller (the library
 *    allocates no device memory). They must be 16-byte aligned.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Calls enqueue work and return; none synchronises the device.
 *  - Return value: ZHA_OK, or a negative zha_status when the host-side checks
 *    reject the arguments (nothing is launched then) or a launch fails
 *    (ZHA_ERR_CUDA). zha_last_error() gives a message for the calling thread.
 *  - Conditions only the device can see are OR-ed into *d_status (int32,
 *    ZHA_DEV_* bits) where the call takes one; the caller zeroes it and reads it
 *    after synchronising.
 *  - Layouts: K and V caches are [n_kv_heads][ld][head_dim] (element type
 *    zha_config.kv_dtype, ld >= tokens used); queries Q are float32
 *    [batch][n_q_heads][head_dim]; query head h uses KV head h / (n_q_heads /
 *    n_kv_heads) [Attention: "Key·value head 를 나눠 쓰거나 압축한다"];
 *    reference queries are float32 [n_kv_heads][n_ref][head_dim].
 *  - No call is thread-safe against another call on the same tree unless the
 *    caller orders them (same stream or events).
 */
#ifndef ZHA_H
#define ZHA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZHA_ABI_VERSION 3

typedef enum {
    ZHA_OK = 0,
    ZHA_ERR_INVALID = -1,     /* bad argument: null pointer, size, alignment, range */
    ZHA_ERR_CAPACITY = -2,    /* a caller buffer (store, workspace, max_sel) is too small */
    ZHA_ERR_STATE = -3,       /* the tree's built prefix does not match n_tokens */
    ZHA_ERR_CUDA = -4,        /* a CUDA launch or query failed (see zha_last_error) */
    ZHA_ERR_UNSUPPORTED = -6  /* a configuration this build does not implement */
} zha_status;

/* Bits OR-ed into *d_status by device code. */
#define ZHA_DEV_SELECTION_TRUNCATED 1 /* zha_route: a head kept more than max_sel chunks; its list holds the first max_sel (ascending) and d_n_chunks the true count */
#define ZHA_DEV_BAD_SELECTION 2       /* zha_sparse_attend: a chunk list had an id out of range, was not strictly ascending, or a count outside [0, max_sel]; out-of-range ids are never read, and which in-range entries of such a list are attended is unspecified */
#define ZHA_DEV_TIMEOUT 4             /* a kernel's bounded wait for its tensor-core work ran out; its outputs are not valid (it released its resources and returned) */
#define ZHA_DEV_BAD_PAGE 8            /* a paged cache's block table named a page outside the pool (or lacked an entry); those keys were not read (treated as absent) and the outputs that needed them are not valid */
#define ZHA_DEV_BAD_LENGTH 16         /* a token count in device memory was outside its range: clamped (zha_attend_batch_kv), or its list item refused (zha_pages_*) */
#define ZHA_DEV_NO_PAGES 32           /* zha_pages_extend / zha_pages_fork: fewer free pages than the call needs; the call changed nothing */
#define ZHA_DEV_BAD_SEQUENCE 64       /* a sequence index out of range, listed twice, or in conflict with another item of its list: that item was refused */

typedef enum { ZHA_F32 = 0, ZHA_BF16 = 1 } zha_dtype;

typedef struct {
    int32_t n_kv_heads;  /* KV heads = trees, >= 1 */
    int32_t n_q_heads;   /* query heads, a multiple of n_kv_heads */
    int32_t head_dim;    /* d: 64 or 128 */
    int32_t chunk;       /* C: tokens per level-1 chunk, 2..128 */
    int32_t levels;      /* L: summary levels, 1..8; level l covers C^l tokens */
    int32_t n_ref;       /* R: reference queries per tree, 1..32 */
    int32_t kv_dtype;    /* zha_dtype of the K and V caches */
    int32_t rope_pairs;  /* rotary positions: 0 = none (position-free keys); else the number
                            of leading element pairs (2i, 2i+1), 1..head_dim/2, that the
                            model turns by position * rope_base^(-2i/head_dim) */
    int64_t max_tokens;  /* tokens the summary store must cover, >= 1 */
    float rope_base;     /* rotation base (> 1) when rope_pairs > 0; ignored otherwise */
    int32_t reserved;    /* must be 0 */
} zha_config;

/* Rotary positions [ZHA: 무엇과 다른가; Attention: "Attention 은 순서를 모르므로 위치
 * 정보를 따로 넣는다"]: with rope_pairs > 0 the caches hold keys as the model
 * rotates them (key of position m turned by m * theta_i per pair i) and decode
 * queries come rotated at their own position. The summaries are then taken at
 * rotated reference queries: node n of level l sits at the position of its
 * first token, p_n = n * C^l, and its reference queries are q_hat_r rotated by
 * p_n. A parent re-evaluates each child c at its own rotated reference query
 * q_hat_{r,P}: u_c = F_c(q_hat_{r,c}) + 1/sqrt(d) <khat_{r,c}, q_hat_{r,P} -
 * q_hat_{r,c}>, which is the child's plane evaluated at q_hat_{r,P}. khat is
 * stored in the keys' (rotated) frame, so routing and attention use the
 * decode queries as they come. */

typedef struct zha_tree zha_tree; /* opaque host handle; holds no device memory */

/* ABI version of the loaded library (ZHA_ABI_VERSION). */
int32_t zha_abi_version(void);

/* Static text for a zha_status. */
const char* zha_status_str(int32_t status);

/* Message describing the last failed call made by the calling thread. */
const char* zha_last_error(void);

/* Number of kernels this library has launched in the process so far. */
uint64_t zha_launch_count(void);

/* Bytes of device memory the summary store of `cfg` needs (0 if cfg is
 * invalid). Layout, level-major: for l = 1..L, float32
 * [n_kv_heads][floor(max_tokens / C^l)][node_floats], each node holding
 * khat [n_ref][head_dim] then bhat [n_ref], padded to node_floats =
 * n_ref*head_dim + round_up(n_ref, 4) [ZHA: 무엇과 다른가]; then, at the next
 * 256-byte boundary, one 256-byte block whose first int32 is the tree's
 * device status word (ZHA_DEV_TIMEOUT set by a build kernel whose bounded wait
 * ran out; zha_build clears it, zha_route passes it on to its d_status).
 * With head_dim 128 and n_ref 16, a second copy of the planes follows, the
 * operand of the tensor-core scoring: for l = 1..L, fp16
 * [n_kv_heads][2][floor(max_tokens / C^l)][n_ref][head_dim], term 0 = khat
 * rounded to fp16 and term 1 = the remainder rounded to fp16. zha_build and
 * zha_append_chunk write it together with the float32 planes; the routing
 * scores from the terms, so a caller that writes planes into the store itself
 * writes their terms as well. */
size_t zha_tree_bytes(const zha_config* cfg);

/* Create a host handle over a caller-owned store (>= zha_tree_bytes bytes,
 * 256-byte aligned) and reference queries d_ref_q [n_kv_heads][n_ref][head_dim]
 * float32, which must stay valid while the tree is used. The tree starts empty
 * (0 tokens built). Returns ZHA_ERR_INVALID / ZHA_ERR_CAPACITY / ZHA_ERR_UNSUPPORTED
 * on bad arguments; *out is set only on success. The learned reference queries
 * are the only trained parameters of the method [ZHA: 어떻게 쓰나]. */
zha_status zha_tree_create(const zha_config* cfg, void* d_store, size_t store_bytes,
                           const float* d_ref_q, zha_tree** out);

/* Release a handle (the store and reference queries stay the caller's). NULL is ignored. */
void zha_tree_destroy(zha_tree* tree);

/* N_b: tokens covered by complete level-1 chunks so far (a multiple of C). */
int64_t zha_tree_built_tokens(const zha_tree* tree);

/* Where level `level` (1..L) lives in the store: float offset of node (g=0,i=0),
 * node capacity per KV head, floats per node. For reading summaries back. */
zha_status zha_tree_level_layout(const zha_tree* tree, int32_t level, int64_t* offset_floats,
                                 int64_t* capacity, int32_t* node_floats);

/* Build every level over the complete chunks of the first n_tokens keys of
 * d_K [n_kv_heads][ld][head_dim] (prefill). Level 1: for chunk i and plane r,
 * s_j = q_r.k_j/sqrt(d) over the chunk, F = LSE_j s_j, khat = sum_j softmax(s)_j k_j,
 * bhat = F - q_r.khat/sqrt(d). Level l >= 2 merges each run of C level-(l-1)
 * nodes: u_c = q_r.khat_{r,c}/sqrt(d) + bhat_{r,c}, F = LSE_c u_c,
 * khat = sum_c softmax(u)_c khat_{r,c}, bhat = F - q_r.khat/sqrt(d)
 * [ZHA: 무엇과 다른가: tangent-plane summary; "parents merge the child summaries
 * in the same way"]. Afterwards N_b = C*floor(n_tokens/C). Requires
 * 0 <= n_tokens <= min(ld, max_tokens). V is not read. The tree's device status
 * word is cleared first; a build kernel whose bounded wait runs out sets
 * ZHA_DEV_TIMEOUT there (its summaries are then not valid), and the next
 * zha_route reports it in its own d_status. */
zha_status zha_build(zha_tree* tree, const void* d_K, int64_t ld, int64_t n_tokens, void* stream);

/* Incremental build while decoding: n_tokens is the cache length after the
 * caller has written the newest keys; the new N_b = C*floor(n_tokens/C) must be
 * >= the tree's N_b (else ZHA_ERR_STATE). Summarises each newly completed chunk
 * and merges every upper-level node the new chunks complete (level 1 every C
 * steps, level 2 every C^2 steps [ZHA: 무엇과 다른가]). One launch when up to
 * 8 chunks are new; a no-op when none is. A time-out of a build kernel is
 * recorded in the tree's device status word as for zha_build. */
zha_status zha_append_chunk(zha_tree* tree, const void* d_K, int64_t ld, int64_t n_tokens,
                            void* stream);

/* Workspace bytes zha_route needs for `batch` queries at n_tokens (grows with
 * n_tokens, so sizing for the largest n_tokens covers smaller ones). */
size_t zha_route_workspace_bytes(const zha_config* cfg, int32_t batch, int64_t n_tokens);

/* uint32 words of the per-level kept bitmaps zha_route can return: level-major
 * for l = 1..L, each [batch][n_q_heads][ceil(n_l / 32)] with n_l =
 * floor(N_b / C^l) nodes at n_tokens; bit i of a head's words = node i kept. */
size_t zha_route_kept_words(const zha_config* cfg, int32_t batch, int64_t n_tokens);

/* Per-level top-p routing of `batch` decode queries d_Q [batch][n_q_heads][d]
 * against the tree at n_tokens (C*floor(n_tokens/C) must equal the tree's N_b,
 * else ZHA_ERR_STATE) [ZHA: 전제와 한계]. For each query head and level L..1:
 * candidates are all level-L nodes at the top, below that the children of the
 * nodes kept one level up plus the level's orphans (nodes whose parent does not
 * exist yet); each candidate n scores sigma_n = max_r (q.khat_{r,n}/sqrt(d) +
 * bhat_{r,n}); pi = softmax(sigma) over the candidates; the kept set is the
 * shortest prefix of the candidates ordered by sigma descending (ties: lower
 * node index first) whose pi sums to >= p; p >= 1 keeps all; 0 < p required.
 * Output: d_chunk_ids [batch][n_q_heads][max_sel] int32, the kept level-1 chunk
 * ids ascending, and d_n_chunks [batch][n_q_heads] their count (the sink and
 * the tail [N_b, n_tokens) are implicit and not listed). d_kept_bits (nullable,
 * zha_route_kept_words words) receives every level's kept bitmap. d_ws:
 * >= zha_route_workspace_bytes bytes. d_status (nullable):
 * ZHA_DEV_SELECTION_TRUNCATED, ZHA_DEV_TIMEOUT (tensor-core scoring, or a
 * build of this tree whose bounded wait ran out, passed on from the tree's
 * status word). */
zha_status zha_route(const zha_tree* tree, const float* d_Q, int32_t batch, int64_t n_tokens,
                     float p, int32_t* d_chunk_ids, int32_t* d_n_chunks, int32_t max_sel,
                     uint32_t* d_kept_bits, void* d_ws, size_t ws_bytes, int32_t* d_status,
                     void* stream);

/* Per-level selection rule of zha_route_ex [ZHA: 전제와 한계]. The pages route
 * with top-p at every level and name its depth scaling: one fixed p per level
 * gives an effective p^L, correcting with p^(1/L) drives p towards 1, so p has
 * to follow depth; they also set top-p against a fixed-budget top-K, which
 * keeps the same number of nodes whether the mass is concentrated or flat. */
typedef enum { ZHA_SELECT_TOP_P = 0, ZHA_SELECT_TOP_K = 1 } zha_select_mode;

typedef struct {
    int32_t mode;      /* zha_select_mode */
    int32_t reserved;  /* must be 0 */
    float p[8];        /* ZHA_SELECT_TOP_P: mass of level l (1..L) at p[l-1]; > 0, finite; >= 1
                          keeps every candidate of that level */
    int32_t k[8];      /* ZHA_SELECT_TOP_K: nodes kept at level l at k[l-1], >= 1: the first
                          min(k, candidates) in the order score descending, node index ascending */
} zha_route_policy;

/* zha_route with a per-level policy: top-p with its own p at each level (for
 * instance p^(1/L) per level), or fixed-budget top-K. Candidates, scores,
 * outputs, workspace and status are as for zha_route; only the cut of each
 * level changes. zha_route(p) is zha_route_ex with mode ZHA_SELECT_TOP_P and p
 * at every level. ZHA_ERR_INVALID for a NULL policy, an unknown mode, reserved
 * != 0, or a p / k of levels 1..L out of range (entries past L are ignored). */
zha_status zha_route_ex(const zha_tree* tree, const float* d_Q, int32_t batch, int64_t n_tokens,
                        const zha_route_policy* policy, int32_t* d_chunk_ids, int32_t* d_n_chunks,
                        int32_t max_sel, uint32_t* d_kept_bits, void* d_ws, size_t ws_bytes,
                        int32_t* d_status, void* stream);

/* Size of the routing scratch built into the library for zha_route_noalloc. */
#define ZHA_ROUTE_NOALLOC_SCRATCH_BYTES (32u << 20) /* 32 MiB per GPU that loads the library */

/* zha_route for callers that cannot allocate device memory. A plugin inside an
 * inference server that owns all device memory may be forbidden to call
 * cudaMalloc; a serving loop with a fixed memory plan cannot allocate per
 * request; a plain C host program may have no device allocator at all. Such
 * callers still pass Q, the outputs, d_kept_bits (nullable) and d_status, as
 * for zha_route, and get the same results, but the scratch zha_route would take
 * as d_ws lives in one fixed device array inside the library
 * (ZHA_ROUTE_NOALLOC_SCRATCH_BYTES, held by every GPU that loads the library
 * until the process exits). This entry point calls no cudaMalloc, cudaFree or
 * other allocating routine.
 *  - A call that needs more scratch than that (zha_route_workspace_bytes, less
 *    the kept bitmaps when d_kept_bits is given) returns ZHA_ERR_CAPACITY and
 *    launches nothing; use zha_route with a workspace then.
 *  - The first call on each device looks up the array's device address (with
 *    that device current) and caches it; make that first call before any
 *    stream capture. With lazy module loading (the CUDA default) that first
 *    lookup is also when the driver loads the library's module on the device
 *    and reserves the array, so a caller whose device memory plan is already
 *    full can see ZHA_ERR_CUDA (out of memory) there: make the first call at
 *    initialisation, before committing the memory plan, or run with eager
 *    module loading (CUDA_MODULE_LOADING=EAGER).
 *  - All calls on a device share the one array and it keeps the last call's
 *    contents (nothing in it needs to start at zero: every call clears or
 *    writes what it reads). Calls whose kernels overlap on the GPU -- on
 *    different streams, or from different threads without ordering -- race on
 *    it; order them.
 * The pages have no counterpart of this call: it only changes where the
 * scratch of zha_route lives. */
zha_status zha_route_noalloc(const zha_tree* tree, const float* d_Q, int32_t batch,
                             int64_t n_tokens, float p, int32_t* d_chunk_ids, int32_t* d_n_chunks,
                             int32_t max_sel, uint32_t* d_kept_bits, int32_t* d_status,
                             void* stream);

/* Workspace bytes zha_sparse_attend needs for `batch` queries at n_tokens. */
size_t zha_attend_workspace_bytes(const zha_config* cfg, int32_t batch, int64_t n_tokens);

/* Exact attention of each query head over S = {0} u tokens(listed chunks) u
 * [N_b, n_tokens), N_b = C*floor(n_tokens/C): o = sum_{j in S} softmax_j(q.k_j/
 * sqrt(d)) v_j, normalised over S only [Attention: "Scaled dot-product attention
 * 의 식"; ZHA: 전제와 한계]. Chunk lists as zha_route writes them (ascending
 * ids < N_b/C, counts <= max_sel); they may also come from elsewhere. The tree
 * supplies only its configuration (its summaries are not read). Output d_O
 * [batch][n_q_heads][d] float32 and, if d_lse is not NULL, d_lse
 * [batch][n_q_heads] = log sum_{j in S} exp(q.k_j/sqrt(d)). d_ws: >=
 * zha_attend_workspace_bytes bytes. d_status (nullable): ZHA_DEV_BAD_SELECTION,
 * ZHA_DEV_TIMEOUT.
 * Requires 1 <= n_tokens <= ld. */
zha_status zha_sparse_attend(const zha_tree* tree, const float* d_Q, const void* d_K,
                             const void* d_V, int64_t ld, int64_t n_tokens, int32_t batch,
                             const int32_t* d_chunk_ids, const int32_t* d_n_chunks,
                             int32_t max_sel, float* d_O, float* d_lse, void* d_ws,
                             size_t ws_bytes, int32_t* d_status, void* stream);

/* ---- Paged K/V caches [Attention: "KV cache 를 담는 방식을 바꾼다: PagedAttention,
 * 양자화"] ---------------------------------------------------------------------
 * A cache held in pages of C tokens (block size = the tree's chunk): a pool
 * [n_pages][C][head_dim] for K and one for V (element type kv_dtype), and a
 * block table: page of chunk c (tokens [cC, (c+1)C)) of KV head g at
 * block_table[g * max_blocks + c]. The in-progress chunk lives in its page too.
 * Summaries, routing and attention are the same as over the contiguous cache
 * holding the same keys and values; only the addresses differ. A table entry
 * outside [0, n_pages) is never dereferenced: ZHA_DEV_BAD_PAGE is set (in the
 * call's d_status, or for builds in the tree's status word, which the next
 * zha_route reports) and those keys count as absent. */
typedef struct {
    const void* k;              /* contiguous: [n_kv_heads][ld][head_dim]; paged: K page pool */
    const void* v;              /* same layout as k; not read by builds (may be NULL there) */
    int64_t ld;                 /* contiguous: token rows per KV head (>= n_tokens); paged: n_pages */
    const int32_t* block_table; /* NULL: contiguous; else [n_kv_heads][max_blocks] int32 page ids */
    int64_t max_blocks;         /* paged: table entries per KV head, >= ceil(n_tokens / C) */
} zha_kv_cache;

/* zha_build / zha_append_chunk / zha_sparse_attend over a zha_kv_cache. The
 * contiguous entry points above are these calls with block_table = NULL. The
 * tensor-core level-1 build serves contiguous caches; paged caches are built
 * by the CUDA-core kernels (same summaries within rounding). */
zha_status zha_build_kv(zha_tree* tree, const zha_kv_cache* kv, int64_t n_tokens, void* stream);
zha_status zha_append_chunk_kv(zha_tree* tree, const zha_kv_cache* kv, int64_t n_tokens, void* stream);
zha_status zha_sparse_attend_kv(const zha_tree* tree, const float* d_Q, const zha_kv_cache* kv,
                                int64_t n_tokens, int32_t batch, const int32_t* d_chunk_ids,
                                const int32_t* d_n_chunks, int32_t max_sel, float* d_O, float* d_lse,
                                void* d_ws, size_t ws_bytes, int32_t* d_status, void* stream);

/* ---- A batch of caches ---------------------------------------------------------
 * The calls below serve n_seqs sequences at once. Their zha_kv_cache holds the
 * caches one behind the other: contiguous [n_seqs][n_kv_heads][ld][head_dim], or
 * paged with a block table [n_seqs][n_kv_heads][max_blocks] over one pool of pages
 * (entries < 0: no page). Sequence s alone is the cache at table row s (or at
 * element s * n_kv_heads * ld * head_dim), as the tree's calls take it. Of the
 * zha_config they read the head counts, head_dim, chunk and kv_dtype; rope_pairs
 * and the tree's own fields must be valid but play no part. At most 2^31 - 512 token
 * slots per pool and 65535 sequences. Arrays lie at multiples of their type's size, or
 * of what a call says; others are refused (ZHA_ERR_INVALID). */

/* ---- Rotary positions [Attention: "Attention 은 순서를 모르므로 위치 정보를 따로
 * 넣는다"] ------------------------------------------------------------------------
 * Pair i of a head is turned by pos * theta_i: (a, b) -> A (a cos - b sin, a sin +
 * b cos), with theta_i = base^(-2i / freq_dim). The elements behind the pairs
 * stay as they are. Angles are kept as 64-bit fractions of a turn, so that a
 * far position loses nothing. A tree with positions (zha_config's rope_pairs) reads keys
 * of one rotation only: INTERLEAVED, PLAIN, pairs = rope_pairs, freq_dim = head_dim, base =
 * rope_base, amplitude 1. Keys turned in any other way are for dense attention, or
 * for a tree with rope_pairs = 0, which takes the cache's keys as they are. */
typedef enum {
    ZHA_ROPE_INTERLEAVED = 0, /* pair i = elements (2i, 2i + 1), the tree's layout (rope_pairs) */
    ZHA_ROPE_HALF = 1         /* pair i = elements (i, i + pairs) */
} zha_rope_layout;

typedef enum {
    ZHA_ROPE_PLAIN = 0,
    ZHA_ROPE_LINEAR = 1, /* theta_i / factor: positions interpolated */
    ZHA_ROPE_NTK = 2,    /* base * factor^(freq_dim / (freq_dim - 2)); freq_dim 2: as LINEAR */
    ZHA_ROPE_YARN = 3,   /* theta_i (1 - w) + theta_i / factor * w, w = clamp((i - lo) / max(hi - lo, 0.001)) to
                            [0, 1], lo = max(0, floor(x(high))), hi = min(freq_dim - 1, ceil(x(low))), x(n) = freq_dim
                            ln(original_tokens / (2 pi n)) / (2 ln base): the pairs that turn more than `high`
                            times over the original length stay, those below `low` turns are
                            interpolated. amplitude 0 stands for 0.1 ln(factor) + 1 */
    ZHA_ROPE_BANDS = 4   /* by turns n = original_tokens theta_i / (2 pi): n >= high stays, n <= low is divided
                            by factor, between them w theta_i + (1 - w) theta_i / factor, w = (n - low) /
                            (high - low) */
} zha_rope_scaling;

typedef struct {
    int32_t head_dim;        /* 64 or 128 */
    int32_t pairs;           /* 1..head_dim/2 turned pairs */
    int32_t layout;          /* zha_rope_layout */
    int32_t scaling;         /* zha_rope_scaling */
    int32_t freq_dim;        /* the exponent's divisor; 0: 2 * pairs (zha_config's rope_pairs uses head_dim) */
    int32_t reserved;        /* must be 0 */
    double base;             /* > 1 */
    double factor;           /* >= 1, read unless PLAIN */
    double original_tokens;  /* > 0, read by YARN and BANDS */
    double low, high;        /* 0 < low < high, read by YARN and BANDS */
    double amplitude;        /* A, >= 0, in the range of float32; 0: 1 (YARN: 0.1 ln(factor) + 1) */
} zha_rope_spec;

/* A rotation ready for use: plain host data, filled by zha_rope_init. */
typedef struct {
    int32_t head_dim, pairs, layout;
    float amplitude;
    uint64_t turn[64]; /* theta_i / (2 pi) as a fraction of 2^64 */
} zha_rope;

zha_status zha_rope_init(const zha_rope_spec* spec, zha_rope* out);

/* Rows of one head each: element e of head h of token t at data + t * token_stride
 * + h * head_stride + e (strides in elements, rows 16-byte aligned). */
typedef struct {
    const void* data;
    int64_t token_stride, head_stride;
} zha_rows;

/* Turn n_heads rows of each of n_tokens tokens at positions d_pos [n_tokens]
 * (int64, any sign). inverse != 0 turns back by the same angles and multiplies
 * by the same amplitude: the transpose, which is the gradient's map from y to x.
 * y (y->data is written) may be x itself with the same type and strides, and must not
 * overlap x otherwise; its rows must lie apart, which is judged by the strides (the
 * smaller spans a row, the larger all rows of the other kind). Types are zha_dtype
 * values; the arithmetic is float32. n_tokens = 0 does nothing. */
zha_status zha_rope_apply(const zha_rope* rope, const zha_rows* x, int32_t x_dtype,
                          const int64_t* d_pos, int64_t n_tokens, int32_t n_heads, int32_t inverse,
                          const zha_rows* y, int32_t y_dtype, void* stream);

/* The new tokens of a batch into its caches: for each of n_new tokens t, key and
 * value rows k, v (n_kv_heads each, element type src_dtype) go to cache row
 * d_index[t] of sequence d_seq[t] in kv_dtype, the keys turned at position
 * d_pos[t] (NULL: d_index), and the query rows q (n_q_heads; NULL: none),
 * turned the same way, to d_q_out [n_new][n_q_heads][head_dim] of type q_dtype,
 * as zha_route, zha_sparse_attend (float32) and zha_attend_batch_kv take them. rope
 * NULL: position-free keys, nothing is turned. kv->k and kv->v are written.
 *  - d_seq[t] < 0: padding; nothing of that token is written (its rows may be read).
 *  - d_seq[t] >= n_seqs, or d_index[t] outside the table or ld: nothing of that token
 *    is written, ZHA_DEV_BAD_SEQUENCE. A table entry outside the pool: that
 *    head's key and value are not written, ZHA_DEV_BAD_PAGE.
 *  - Two tokens with the same sequence and index, or whose sequences share that
 *    page, leave either's values there (per element); zha_pages_fork keeps
 *    part-filled pages apart for this reason.
 * d_q_out must not overlap the inputs. n_new = 0 does nothing. */
zha_status zha_rope_append_kv(const zha_config* cfg, const zha_rope* rope, const zha_rows* q,
                              const zha_rows* k, const zha_rows* v, int32_t src_dtype, int64_t n_new,
                              const zha_kv_cache* kv, int32_t n_seqs, const int32_t* d_seq,
                              const int64_t* d_index, const int64_t* d_pos, void* d_q_out,
                              int32_t q_dtype, int32_t* d_status, void* stream);

/* ---- Dense attention of a batch [Attention: "FlashAttention 계열"] -----------------
 * One query token per sequence over all of its keys: o = sum_{j < n} softmax_j(q.k_j /
 * sqrt(d)) v_j with n = d_n_tokens[s] (int64, in device memory), query head h on KV head
 * h / (n_q_heads / n_kv_heads). The dense arm of the decode step, for short
 * contexts, which routing does not pay for, and to measure routing against. d_Q and
 * d_O [n_seqs][n_q_heads][head_dim] have type q_dtype (float32 or bf16) and may be one
 * buffer, but must not overlap otherwise; d_lse (nullable) float32 [n_seqs][n_q_heads]. n = 0, or no page of the sequence
 * in the pool: o = 0, lse = -inf. A count outside [0, max_tokens] is clamped
 * (ZHA_DEV_BAD_LENGTH). Keys whose table entry is outside the pool count as
 * absent (ZHA_DEV_BAD_PAGE). Rows behind n are not read. Requires max_tokens <= ld, or
 * <= max_blocks * C. The split over the cache is made on the device from the counts,
 * so a captured call may be replayed with other counts. The workspace holds
 * nothing between calls; calls that may overlap need one each. For finite inputs a
 * float32 result has the error of float32 sums: over a bf16 cache every operand enters
 * exactly, over a float32 cache within 2^-22; with bf16 queries weights enter within
 * 2^-16. An infinity or NaN in a query or key makes the output and lse of its own
 * heads and sequence NaN, one in a value its own element of their outputs infinite or
 * NaN, and no others. (A finite key whose score passes the range of float32
 * downwards has a weight of 0, as in the formula.) */
size_t zha_attend_batch_workspace_bytes(const zha_config* cfg, int32_t n_seqs, int64_t max_tokens);
zha_status zha_attend_batch_kv(const zha_config* cfg, const void* d_Q, int32_t q_dtype,
                               const zha_kv_cache* kv, int32_t n_seqs, const int64_t* d_n_tokens,
                               int64_t max_tokens, void* d_O, float* d_lse, void* d_ws,
                               size_t ws_bytes, int32_t* d_status, void* stream);

/* ---- Pages of a batch [Attention: "KV cache 를 담는 방식을 바꾼다: PagedAttention,
 * 양자화"] ------------------------------------------------------------------------
 * Which pages are in use is the pool's reference counts, in device memory: refs[p] =
 * the table entries that name page p, 0 = free. The calls run on the device alone
 * (capturable) and always hand out the lowest free pages, in the order item, KV head,
 * block, so that a run can be repeated exactly. Lists are int32 [n_items] sequence
 * indexes with int64 token counts. An item of extend or fork whose index is out of
 * range or already listed is refused (ZHA_DEV_BAD_SEQUENCE), one whose count is negative or
 * does not fit in max_blocks pages too (ZHA_DEV_BAD_LENGTH); the others go ahead. Free
 * says below what it refuses. n_items = 0 does nothing. Calls on one pool need an order (a stream) between them. */
typedef struct {
    void* k;                /* K pool [n_pages][C][head_dim] */
    void* v;                /* V pool, the same shape */
    int64_t n_pages;
    int32_t* block_table;   /* [n_seqs][n_kv_heads][max_blocks], < 0: no page */
    int64_t max_blocks;
    int32_t* refs;          /* [n_pages] */
    int32_t n_seqs;
    int32_t reserved;       /* must be 0 */
} zha_page_pool;

/* Workspace of zha_pages_extend, _fork (n_items) and _compact (n_items = 0); holds
 * nothing between calls. */
size_t zha_pages_workspace_bytes(const zha_config* cfg, const zha_page_pool* pool, int32_t n_items);

/* A page for every block without one among the first ceil(d_n_tokens[i] / C) blocks of
 * each KV head of sequence d_seqs[i]. An item with an entry among them that names no
 * page in use is refused (ZHA_DEV_BAD_PAGE). All other items or, when the free
 * pages do not suffice, none (ZHA_DEV_NO_PAGES). */
zha_status zha_pages_extend(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_seqs,
                            const int64_t* d_n_tokens, int32_t n_items, void* d_ws, size_t ws_bytes,
                            int32_t* d_status, void* stream);

/* Sequence d_dst[i] becomes a copy of the first d_n_tokens[i] tokens of d_src[i]:
 * full pages are shared (refs + 1), the rows in use of a part-filled last page are
 * copied to a page of its own, whose other rows stay as they were. One source may
 * serve many items. Refused are an item whose destination is not empty (all entries
 * < 0) or whose source is a destination of the same list (ZHA_DEV_BAD_SEQUENCE), and one
 * whose source lacks a page in use for its tokens (ZHA_DEV_BAD_PAGE). All other items
 * or, without enough free pages, none (ZHA_DEV_NO_PAGES). */
zha_status zha_pages_fork(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_src,
                          const int32_t* d_dst, const int64_t* d_n_tokens, int32_t n_items, void* d_ws,
                          size_t ws_bytes, int32_t* d_status, void* stream);

/* Give up the blocks from ceil(d_keep[i] / C) on (d_keep NULL: all blocks) of
 * sequence d_seqs[i]: refs - 1, entry -1; a page at 0 is free. A sequence listed twice
 * keeps the smaller count, and one whose count is more than max_blocks pages hold
 * keeps all that it has; a negative count is refused (ZHA_DEV_BAD_LENGTH). An entry that names no page in use is cleared
 * (ZHA_DEV_BAD_PAGE). Cut back inside a shared page, a sequence must not be
 * written there: fork it first. */
zha_status zha_pages_free(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_seqs,
                          const int64_t* d_keep, int32_t n_items, int32_t* d_status, void* stream);

/* Pack the pool: with n pages in use, the k-th of them at or above n moves
 * (contents, count, table entries of all sequences) to the k-th free page below n,
 * so that pages [0, n) are the ones in use. d_page_map (nullable) int32 [n_pages]:
 * the new place of each page that was in use, -1 of a free one; d_n_live
 * (nullable) int32: n. A table entry that names a free page becomes -1
 * (ZHA_DEV_BAD_PAGE); one outside the pool stays. */
zha_status zha_pages_compact(const zha_config* cfg, const zha_page_pool* pool, int32_t* d_page_map,
                             int32_t* d_n_live, void* d_ws, size_t ws_bytes, int32_t* d_status,
                             void* stream);

/* ---- Routing diagnostics [ZHA: 어떻게 쓰나; 전제와 한계] -----------------------
 * How well each level's estimate follows the dense attention mass, for
 * `batch` queries d_Q [batch][n_q_heads][d] against the tree and the keys d_K
 * [n_kv_heads][ld][d] at n_tokens (the tree must cover C*floor(n_tokens/C),
 * else ZHA_ERR_STATE). For every level l and query head:
 *   target p_{l}(n) = the dense softmax weights of q over the keys the level's
 *     complete nodes cover, summed node by node (the reference queries' KL
 *     training target [ZHA: 어떻게 쓰나]; the in-progress tail is in no node);
 *   estimate p_hat_{l}(n) = softmax over the level's nodes of max_r t_r(q);
 *   d_kl[l-1][batch][n_q_heads] = KL(p_l || p_hat_l) (float32, natural log).
 * d_usage (nullable, uint32 [L][n_ref], ACCUMULATED -- the caller zeroes it):
 * for every node of every level and every query head, +1 at the plane r that
 * gives the node's score (lowest r on ties); [ZHA: 전제와 한계] reports that
 * few reference queries serve the upper levels and that their use evens out
 * towards the leaves. Every node of every level is scored and the dense mass of
 * every complete chunk is formed, so this costs a dense pass over the keys: a
 * diagnostic, not part of routing. d_ws: >= zha_diagnostics_workspace_bytes. */
size_t zha_diagnostics_workspace_bytes(const zha_config* cfg, int32_t batch, int64_t n_tokens);
zha_status zha_route_diagnostics(const zha_tree* tree, const float* d_Q, const void* d_K, int64_t ld,
                                 int32_t batch, int64_t n_tokens, float* d_kl, uint32_t* d_usage,
                                 void* d_ws, size_t ws_bytes, void* stream);

/* ---- Test hook (the pages have no counterpart) ------------------------------
 * For tests of the bounded waits of this tree's tensor-core level scoring
 * (head_dim 128, R = 16): wait_polls = polls of each of its mbarrier waits
 * before the wait gives up (0 restores the default, about 2 s; each poll lets
 * the thread sleep up to about 65 us); withhold != 0 makes its producer send
 * nothing, so that the consumers' waits run out with nothing in flight: the
 * kernel releases its tensor memory, returns, and the route reports
 * ZHA_DEV_TIMEOUT (its outputs are then not valid). Not for production use. */
zha_status zha_tree_debug(zha_tree* tree, uint32_t wait_polls, int32_t withhold);

/* ---- Kernel timing (profiling; the pages have no counterpart) ------------
 * While enabled, every kernel the library launches whose name contains
 * `name_filter` (NULL or "" = all) and whose tag equals `tag_filter` (-1 = all;
 * the tag is the tree level for the routing kernels, 0 otherwise) is bracketed
 * by two CUDA events recorded on its stream. Up to `max_records` launches are
 * recorded (later ones are counted as dropped); max_records <= 0 disables
 * tracing. The events are created here (host-side driver objects, no device
 * memory); each enable discards the previous records. Recording events between
 * kernels removes their programmatic overlap, so traced calls run a little
 * slower than untraced ones. Not thread-safe against concurrent launches from
 * other threads while enabled. */
zha_status zha_trace_enable(int32_t max_records, const char* name_filter, int32_t tag_filter);

/* Launches recorded since the last enable or clear, and launches dropped
 * because the records were full. */
int32_t zha_trace_count(void);
int32_t zha_trace_dropped(void);

/* Record i (0 <= i < zha_trace_count()): kernel name (static string), tag and
 * device time in milliseconds. The caller must have synchronised the streams
 * the kernels ran on. */
zha_status zha_trace_read(int32_t i, const char** name, int32_t* tag, float* ms);

/* Forget the records (the events are kept for reuse). */
void zha_trace_clear(void);

#ifdef __cplusplus
}
#endif

#endif /* ZHA_H */
