/*
 * saf3r.h - C ABI of the head-wise dynamic sparse global attention library.
 *
 * The method is SAF3R ("SAF3R: Dynamic Sparse Attention for Feed-Forward 3D
 * Reconstruction Transformers", arXiv 2607.03612).  Every attention head of a
 * cross-view global-attention layer gets its own key/value index set, chosen
 * by one of four kernels (section 4.1): a static position/anchor pattern, a
 * mean-query-probe Top-K (vertical-line heads), a DINO-feature Top-K
 * (correspondence heads) or a uniform stride (scanning heads).  Exact softmax
 * attention then runs over the kept keys only; the dynamic sets are built once
 * per input and cached (section 4.3); an offline step picks each head's
 * configuration from the output NMSE against full attention (section 4.2).
 *
 * Conventions shared by every call
 *   - Token layout: S views; each view holds n_special special tokens
 *     (camera, registers) followed by grid_h*grid_w patch tokens in raster
 *     order.  V = n_special + grid_h*grid_w, N = S*V, token t = s*V + i.
 *   - Q, K, V, O are row-major [H][N][d] tensors (bf16 inputs; bf16 or fp32
 *     output), d = 64, rows of 128 bytes.  DINO features are fp32
 *     [S*grid_h*grid_w][dino_dim], one row per patch token in token order.
 *   - All pointers named q, k, v, dino, out, cache and workspace are DEVICE
 *     pointers, 16-byte aligned.  `stream` is a cudaStream_t (NULL = legacy
 *     default stream).  The caller owns every buffer; the library allocates
 *     no device memory and keeps no state except one error word per device.
 *   - Calls are asynchronous on `stream` unless stated.  Argument errors are
 *     returned at once and launch nothing.  Errors found on the device (a
 *     bounded wait that expired, an index cache built for another layout)
 *     are recorded in the device error word and reported by saf3r_check().
 *   - Attention scale is 1/sqrt(d); excluded keys take no part in the softmax
 *     (their logit is -inf), so each row is an exact softmax over its kept set.
 */
#ifndef SAF3R_H
#define SAF3R_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SAF3R_OK = 0,
    SAF3R_ERR_INVALID = 1,      /* bad argument, or cache/layout mismatch found on the device */
    SAF3R_ERR_CUDA = 2,         /* a CUDA runtime/driver call failed */
    SAF3R_ERR_TIMEOUT = 3,      /* a bounded device wait expired; the kernel gave up cleanly */
    SAF3R_ERR_INDEX = 4,        /* an index read from the cache was out of range */
    SAF3R_ERR_UNSUPPORTED = 5   /* shape or device not supported (d != 64, not sm_100) */
} saf3r_status;

/* Head kinds (section 3, Observation #2; kernels of section 4.1). */
typedef enum {
    SAF3R_POSITION = 0,  /* static kernel: specials + anchor view 0 + the 3x3 cell neighbourhood in every view */
    SAF3R_PROBE = 1,     /* query-probe Top-K: Top-k patch keys by mean-query score, + all specials */
    SAF3R_CORR = 2,      /* DINO Top-K, block-wise: per 64-query tile, Top-k 64-token key tiles + all specials */
    SAF3R_SCAN = 3,      /* uniform sampling: keys j with j mod stride == phase, + all specials */
    SAF3R_DENSE = 4,     /* every key (full attention) */
    SAF3R_HYBRID = 5,    /* CORR's k key tiles united with SCAN's lattice (stride, phase), + all specials:
                            the Top-K / uniform-stride combination that section 5.3 ("Further Analysis
                            of the DINO Top-K kernel") proposes against regions the DINO matches miss */
    SAF3R_TOKEN = 6      /* DINO Top-K, token-wise: a patch query keeps, in every frame, the k patch tokens of
                            highest DINO cosine (section 4.1; section 5.1 sets k per frame), + all specials;
                            a special-token query (no DINO feature) keeps every key */
} saf3r_head_type;

typedef struct {
    int32_t S;          /* views, >= 1 */
    int32_t grid_h;     /* patch rows per view */
    int32_t grid_w;     /* patch columns per view */
    int32_t n_special;  /* special tokens per view (5: 1 camera + 4 registers) */
    int32_t H;          /* heads, 1..64 */
    int32_t d;          /* head dimension; must be 64 */
    int32_t dino_dim;   /* DINO feature width (384); 1..1024 */
    int32_t tile;       /* token tile of the block-wise DINO kernel; must be 64 */
} saf3r_layout;

typedef struct {
    int32_t type;       /* saf3r_head_type */
    int32_t k;          /* PROBE: kept patch keys (1..S*grid_h*grid_w); CORR, HYBRID: kept key tiles (1..T);
                           TOKEN: kept patch tokens per frame (1..grid_h*grid_w) */
    int32_t stride;     /* SCAN, HYBRID: >= 1 */
    int32_t phase;      /* SCAN, HYBRID: 0 <= phase < stride */
    int32_t radius;     /* POSITION: neighbourhood radius in cells, 0..3 (1 = 3x3); -1 = the anchor frame
                           only (section 4.1's first static example: all queries attend to view 0) */
} saf3r_head_cfg;

/* Operations for saf3r_workspace_bytes. */
enum { SAF3R_OP_SELECT = 0, SAF3R_OP_SPARSE = 1, SAF3R_OP_DENSE = 2, SAF3R_OP_PROFILE = 3 };

/*
 * Size in bytes of the index cache that saf3r_select_kv fills for this layout
 * and per-head configuration (cfg: H entries).  The cache holds a header with
 * a hash of (layout, cfg), each probe head's kept patch keys (int32, ascending)
 * and, if any head is CORR or HYBRID, the ranked key-tile list of every query
 * tile (int32 [T][kmax], best first; T = ceil(N/64), kmax = largest such k),
 * and, if any head is TOKEN, the ranked per-frame lists of every patch query
 * (int32 [S*P][S][kmax] patch indices, best first; kmax = largest TOKEN k),
 * and, where the layout allows (S*P patches, P up to about 6,000, at most
 * 2^28 union entries per budget), the patch queries' order for the tensor
 * cores plus, per distinct TOKEN k and per 256 queries of that order, room
 * for the union of their kept tokens (S * min(256 k, P) entries, int32) and
 * one 64-bit mask per query and 64 union entries: about
 * 36 * ceil(S*P/256) * S * min(256 k, P) bytes per distinct k (2.6 GB at
 * S = 100, P = 1369, k = 16).
 * Returns 0 for an invalid layout or cfg.
 */
size_t saf3r_cache_bytes(const saf3r_layout* layout, const saf3r_head_cfg* cfg);

/*
 * Size in bytes of the device workspace that operation `op` needs:
 * SAF3R_OP_SELECT or SAF3R_OP_SPARSE with the per-head cfg (H entries),
 * SAF3R_OP_DENSE with cfg = NULL.  Profiling uses
 * saf3r_profile_workspace_bytes.  Returns 0 for invalid arguments.
 */
size_t saf3r_workspace_bytes(const saf3r_layout* layout, const saf3r_head_cfg* cfg, int op);

/* Workspace bytes of saf3r_profile_heads for n_cand candidates. */
size_t saf3r_profile_workspace_bytes(const saf3r_layout* layout, const saf3r_head_cfg* cand, int n_cand);

/*
 * Build the per-input dynamic index sets (section 4.3, "Online Pattern
 * Adaptation") and write them to `cache` (saf3r_cache_bytes bytes).
 *   - PROBE heads: qbar = mean of all N query rows of the head (fp64 sum,
 *     rounded once to fp32); score_j = qbar . k_j / sqrt(d) in fp32; the k
 *     patch keys of highest score (ties to the lower token index) are kept.
 *     Section 4.3 shows this ranking equals ranking keys by the column means
 *     of Q K^T / sqrt(d).
 *   - CORR heads: each flat 64-token tile gets the mean of the L2-normalised
 *     DINO features of its patch tokens; tiles are compared by cosine; every
 *     query tile ranks all tiles (itself included; ties to the lower tile).
 *     Computed once and shared by all CORR and HYBRID heads (prefixes serve
 *     smaller k).
 *   - TOKEN heads: L2-normalised DINO features; for every patch query and
 *     every frame, the frame's patch tokens ranked by cosine (own token
 *     included; ties to the lower patch index); the lists are cached.
 *     The cosines are formed on the tensor cores (fp16 features, fp32
 *     accumulation, fp16 scores: within 2e-3 of the exact cosine) and every
 *     candidate within twice that bound of the k-th score is recomputed
 *     exactly (fp64), so the ranking is that of the fp64 cosines rounded to
 *     fp32.  The workspace then holds the fp16 scores of up to 1 GiB of query
 *     rows at a time.  Needs dino_dim <= 384 (SAF3R_ERR_UNSUPPORTED otherwise).
 *     The patch queries are then ordered by their best match in frame 0,
 *     then in frame 1 (queries that see the same scene point become
 *     neighbours), and every 256 queries of that order get the ascending
 *     union of their kept tokens and a per-query bitmask over it, which the
 *     attention streams through the tensor cores.
 *   - POSITION, SCAN and DENSE heads need no cached state (a HYBRID head's
 *     lattice neither).
 * q, k: bf16 [H][N][d]; dino: fp32 patch features, or NULL when no head is
 * CORR, HYBRID or TOKEN.
 * workspace: saf3r_workspace_bytes(layout, cfg, SAF3R_OP_SELECT) bytes.
 */
saf3r_status saf3r_select_kv(const saf3r_layout* layout, const saf3r_head_cfg* cfg,
                             const void* q, const void* k, const float* dino,
                             void* cache, void* workspace, void* stream);

/*
 * saf3r_select_kv without a caller workspace.  No counterpart in the paper: this
 * entry point exists for callers that cannot allocate device memory for the
 * workspace - engines whose latency-critical loop must not enter an allocator,
 * plug-in hosts that pass a library only its inputs and outputs.  It builds
 * exactly the cache saf3r_select_kv builds, taking its scratch from a 40 MiB
 * device array compiled into the library (held by every GPU that loads the
 * library until the process exits), and calls no allocator.
 *   - Limit: saf3r_workspace_bytes(layout, cfg, SAF3R_OP_SELECT) must be at most
 *     40 MiB (41943040 bytes; the 274,800-token layer with 4 probe and 4
 *     correspondence heads needs 32.3 MiB); larger layers return
 *     SAF3R_ERR_UNSUPPORTED and launch nothing.
 *   - First-call setup: the first call on each device looks up the array's
 *     device address (cudaGetSymbolAddress) and remembers it; later calls on
 *     that device reuse it.
 *   - All calls share the one array: calls that may overlap on the GPU (other
 *     streams, other host threads) race and must be serialised by the caller.
 *     Nothing in the array needs to start at zero; each call clears what it needs.
 * Arguments and errors as saf3r_select_kv.
 */
saf3r_status saf3r_select_kv_static(const saf3r_layout* layout, const saf3r_head_cfg* cfg,
                                    const void* q, const void* k, const float* dino,
                                    void* cache, void* stream);

/*
 * Sparse global attention over cached index sets (section 4.1): for every head
 * h and query i, O[h][i] = sum_{j in kept(h,i)} softmax_j(q.k_j/sqrt(d)) v_j.
 * `cache` must come from saf3r_select_kv with the same layout and cfg (checked
 * on the device through the cache header hash; a mismatch records
 * SAF3R_ERR_INVALID and leaves `out` unwritten).  q, k, v may be fresh
 * tensors of a later layer call: the cached sets are reused as they are.
 * All heads run in one tensor-core launch; a TOKEN head's patch queries run
 * there over their cached per-256-query key unions (each query masked to its
 * own keys) when the layout has unions and the launch's per-head plans fit
 * (at most 64 plans: one per head, plus one per TOKEN head with special
 * tokens), else in a per-query gather kernel.  Both give the exact softmax
 * over each query's kept keys.
 * out: bf16 [H][N][d] (out_is_fp32 = 0) or fp32 (out_is_fp32 = 1).
 * workspace: saf3r_workspace_bytes(layout, cfg, SAF3R_OP_SPARSE) bytes.
 */
saf3r_status saf3r_sparse_attn(const saf3r_layout* layout, const saf3r_head_cfg* cfg, const void* cache,
                               const void* q, const void* k, const void* v,
                               void* out, int out_is_fp32, void* workspace, void* stream);

/*
 * Full attention over all N keys for every head: O_full of section 4.2, the
 * reference of the per-head NMSE.  Layout arguments as saf3r_sparse_attn.
 * workspace: saf3r_workspace_bytes(layout, NULL, SAF3R_OP_DENSE) bytes.
 */
saf3r_status saf3r_dense_attn(const saf3r_layout* layout, const void* q, const void* k, const void* v,
                              void* out, int out_is_fp32, void* workspace, void* stream);

/*
 * Offline head profiling (section 4.2) on one calibration input.  For every
 * candidate c (n_cand entries; a SCAN candidate's phase is replaced by
 * head mod stride) and every head h it computes
 *     nmse[h*n_cand + c]  = ||O_full - O_c||^2 / ||O_full||^2        (eq. 1)
 *     pairs[h*n_cand + c] = number of (query, kept key) pairs (Omega = 4*d*pairs)
 * and chooses for each head the candidate of least Omega whose NMSE is at
 * most nmse_max (ties to the lower candidate index); when none qualifies, the
 * candidate of least NMSE (the argmin of eq. 2).  chosen (H entries), nmse
 * and pairs are HOST arrays.  Synchronizes `stream`.
 * workspace: saf3r_profile_workspace_bytes(layout, cand, n_cand) bytes.
 */
saf3r_status saf3r_profile_heads(const saf3r_layout* layout, const saf3r_head_cfg* cand, int n_cand,
                                 const void* q, const void* k, const void* v, const float* dino,
                                 double nmse_max, saf3r_head_cfg* chosen, double* nmse, int64_t* pairs,
                                 void* workspace, void* stream);

/*
 * The search of section 4.2, eq. 2 ("progressive local substitution"), as a
 * host-side rule over the tables saf3r_profile_heads measured on each input
 * of a calibration set.  Per head h and candidate c it averages eq. 1 over
 * the n_inputs inputs (E[h][c], fp64 sum in input order / n_inputs) and the
 * kept pairs likewise (W[h][c], the cost: Omega = 4*d*pairs, so comparisons of
 * pairs are comparisons of Omega).  Then, per head, it starts from the
 * baseline candidate `base` (the uniform-stride SCAN candidate at the target
 * sparsity sigma: stride ceil(1 / (1 - sigma))) and visits the other
 * candidates in index order, making c the current choice when
 * W[h][c] <= W[h][base] and E[h][c] < E[h][current].  The result minimises the
 * error under the baseline's cost; ties go to the baseline, then to the lower
 * candidate index.
 *
 * nmse:  HOST double  [n_inputs][H][n_cand] (saf3r_profile_heads' nmse, per input)
 * pairs: HOST int64   [n_inputs][H][n_cand] (saf3r_profile_heads' pairs, per input)
 * choice: HOST int32  [H] out, the chosen candidate index per head
 * nmse_mean: HOST double [H][n_cand] out (E), or NULL
 * Returns SAF3R_ERR_INVALID for null inputs, n_inputs, H or n_cand < 1, or
 * base out of range.  No device work, no stream.
 */
saf3r_status saf3r_choose_eq2(int n_inputs, int H, int n_cand, const double* nmse, const int64_t* pairs,
                              int base, int32_t* choice, double* nmse_mean);

/*
 * Stride of the uniform-sampling baseline from which the eq. 2 search starts
 * (section 4.2: uniform sampling at sparsity ratio sigma; section 5.1 uses
 * sigma = 0.85): keeping one key in s has sparsity 1 - 1/s, so the baseline
 * stride is the smallest s with 1 - 1/s >= sigma, i.e. ceil(1 / (1 - sigma))
 * (7 for sigma = 0.85).  Returns -1 for sigma outside [0, 1).  Host only.
 */
int32_t saf3r_baseline_stride(double sigma);

/*
 * Copy one head's cached index list to host memory (synchronizes `stream`):
 * PROBE head -> its k kept patch keys (ascending); CORR or HYBRID head -> the
 * ranked tile list int32 [T][k] truncated to that head's k; TOKEN head -> the
 * per-frame lists int32 [S*P][S][k] (patch indices) truncated to its k.  *n receives the number
 * of entries; at most `cap` are written.  Other head kinds return
 * SAF3R_ERR_INVALID.
 */
saf3r_status saf3r_cache_export(const saf3r_layout* layout, const saf3r_head_cfg* cfg, const void* cache,
                                int head, int32_t* host_idx, size_t cap, size_t* n, void* stream);

/*
 * Exact number of (query, kept key) pairs of every head under (layout, cfg)
 * with the index sets held in `cache` (section 4.2: the cost of a
 * configuration is Omega = 4*d*pairs FLOPs).  pairs: HOST int64 [H].
 * Synchronizes `stream` (the correspondence heads' tile lists are read back).
 */
saf3r_status saf3r_kept_pairs(const saf3r_layout* layout, const saf3r_head_cfg* cfg, const void* cache,
                              int64_t* pairs, void* stream);

/* ====================================================================== views taken one after another
 *
 * Streaming: the tokens of new views are rotated by their positions, their keys and values are
 * appended to a paged cache, and their queries attend to the cached tokens.  No counterpart in the
 * paper, which has all views in hand.  d = 64 throughout.
 *
 * Strides are in elements; a row's 64 values are contiguous.  Row starts must be 16-byte aligned
 * (base pointers, and token and head strides a multiple of 8 for bf16 tensors, of 4 for fp32 ones).
 * Strides may be in any order (token-major or head-major), but not negative; rows of queries and outputs may not overlap
 * one another.  Calls whose output shares bytes with what they read are refused (SAF3R_ERR_INVALID), but for rotation in
 * place.  Rows of one packed buffer may interleave where their token strides are equal (in bytes) or their ranges lie apart.
 */

/* How the rotated dims of a head pair up. */
typedef enum {
    SAF3R_ROPE_HALF = 0,     /* each axis has its own dims[a] consecutive dims (axis 0 first), D = dims[a]:
                                dims i and i + D/2 of them turn by pos[a] * base^(-2i/D) */
    SAF3R_ROPE_PAIRS = 1,    /* the same, dims 2i and 2i + 1 */
    SAF3R_ROPE_SECTIONS = 2  /* one rotation over the whole width R = sum of dims: dims j and j + R/2 turn by
                                pos[axis(j)] * base^(-2j/R), the first dims[0]/2 values of j being axis 0's,
                                the next dims[1]/2 axis 1's, and so on */
} saf3r_rope_pairing;

/* Rotary positions with several axes ((row, column) of images; (time, row, column) of videos).  A
 * pair (a, b) that turns by the angle x becomes (a cos x - b sin x, a sin x + b cos x).  Dims from
 * the sum of dims on are not rotated. */
typedef struct {
    int32_t n_axes;     /* 1..4 */
    int32_t pairing;    /* saf3r_rope_pairing */
    int32_t dims[4];    /* rotated dims of each axis: multiples of 8, >= 8; their sum at most 64 */
    double base;        /* frequency base, 1 <= base <= 1e12 */
} saf3r_rope_cfg;

/*
 * Rotate the first n_rot_heads heads of x by the tokens' positions and copy the others.
 *   x, out: n_tokens x n_heads rows of 64 (bf16, or fp32 where *_is_fp32), rows of token t and head h at
 *           t * token_stride + h * head_stride; out may be x itself (same type and strides), no
 *           other overlap.  A projection's packed [token][q, k, v][head][64] rows are 3H heads of
 *           which 2H are rotated, and head-major out strides give the [H][N][64] rows that the
 *           attention calls take.
 *   pos:    DEVICE int32 [n_tokens][n_axes], any value
 *   inverse: nonzero turns by minus the angle: the adjoint, so the gradient of x from that of out
 * Angles are worked out in 64-bit fixed point, to 2^-33 turns at every int32 position, and rounded to
 * fp32 as a part of the nearest quarter turn (2^-28 turns at most); the rotation is in fp32 and rounded once.
 */
typedef struct {
    int64_t n_tokens;
    int32_t n_heads, n_rot_heads;
    const void* x;
    int64_t x_token_stride, x_head_stride;
    void* out;
    int64_t out_token_stride, out_head_stride;
    int32_t x_is_fp32, out_is_fp32;
    const int32_t* pos;
    int32_t inverse;
} saf3r_rope_args;
saf3r_status saf3r_rope(const saf3r_rope_cfg* rope, const saf3r_rope_args* args, void* stream);

/* Element types of a key/value cache. */
typedef enum {
    SAF3R_KV_BF16 = 0,
    SAF3R_KV_E4M3 = 1   /* 8-bit floating point (4 exponent, 3 mantissa bits, largest 448); a value is
                           code * scale, one fp32 scale for each (page, kv head) of keys and of values */
} saf3r_kv_type;

/*
 * A paged cache of keys and values, in DEVICE memory of the caller: pools [n_pages][n_heads][page][64]
 * and, for SAF3R_KV_E4M3, scales fp32 [n_pages][n_heads], always a power of two in 2^-100 .. 2^119.
 * Nothing needs a start value.  Pools and scales 16-byte aligned.
 */
typedef struct {
    int32_t n_pages;    /* >= 1 */
    int32_t n_heads;    /* key/value heads, 1..64 */
    int32_t page;       /* tokens of a page: 16, 32, 64 or 128 */
    int32_t type;       /* saf3r_kv_type */
    void* k;
    void* v;
    float* k_scale;     /* NULL for SAF3R_KV_BF16 */
    float* v_scale;
} saf3r_kv_cache;

/*
 * The new tokens of one step of several sequences (streams).  Sequence b has
 * new = cu_tokens[b+1] - cu_tokens[b] new tokens: rows cu_tokens[b].. of the step's tensors, and
 * tokens kv_lens[b] - new .. kv_lens[b] - 1 of the sequence.  Token i of it lives in row i % page of
 * page page_table[b][i / page].  Arrays are DEVICE int32, read by the kernels: a captured graph
 * follows their contents.  Rows behind the last sequence are not touched.  A sequence whose numbers
 * do not fit (new < 0 or > max_new, rows outside 0 .. n_tokens, kv_lens > max_pages * page, kv_lens < new) or
 * that needs a page outside the cache records SAF3R_ERR_INDEX: nothing is read or written outside the
 * buffers, that sequence's results are unspecified (where cu_tokens runs back, those of sequences behind it too).
 */
typedef struct {
    int32_t n_seqs;     /* 0..65535 */
    int32_t n_tokens;   /* rows of the step's tensors, >= 0 */
    int32_t max_new;    /* the most new tokens of one sequence (a bound, for the launch), 0..n_tokens */
    int32_t max_pages;  /* entries of a sequence's row of page_table */
    const int32_t* cu_tokens;   /* [n_seqs + 1] */
    const int32_t* kv_lens;     /* [n_seqs], with the new tokens */
    const int32_t* page_table;  /* [n_seqs][max_pages]; entries of pages that no call needs may be anything */
} saf3r_kv_batch;

/* Key and value rows of a step: bf16, n_tokens x n_heads rows of 64. */
typedef struct {
    const void* k;
    int64_t k_token_stride, k_head_stride;
    const void* v;
    int64_t v_token_stride, v_head_stride;
    const int32_t* pos;   /* [n_tokens][n_axes] with a rope, else NULL */
} saf3r_kv_rows;

/*
 * Append the new tokens' keys and values to the cache.
 *   rope: keys are rotated on the way (fp32, rounded once to the cache's type; for SAF3R_KV_E4M3 scales and codes are
 *     those of the exact rotation, to its angle's 2^-33 turns); NULL: as they are.
 *   SAF3R_KV_E4M3: of each (page, head), keys and values apart, the scale becomes
 *     2^ceil(log2(m / 448)), m the largest finite magnitude among the new rows, but at least 2^-100, and not
 *     less than the scale of the page's older rows when it has any; where that grew, the older rows' codes are
 *     rounded again to the new scale (exact but for codes that become subnormal).  Codes are rounded to nearest,
 *     ties to even; infinities and NaN become NaN.
 * A page may take new rows of one sequence only, and once in its row of page_table; pages shared by sequences must be full.
 */
saf3r_status saf3r_kv_append(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch,
                             const saf3r_rope_cfg* rope, const saf3r_kv_rows* rows, void* stream);

/*
 * Which tokens a query sees.  Tokens form views of view_tokens tokens in order (view_tokens 1: every token
 * is its own view).  A query of view f sees
 *   causal:      the views f - window + 1 .. f, and of the views 0 .. f the first n_sink tokens
 *   not causal:  the views f - window + 1 .. f + window - 1, and the first n_sink tokens
 * window 0: all views on those sides.  A token out of sight takes no part, whatever it holds.
 */
typedef struct {
    int32_t view_tokens;  /* >= 1 */
    int32_t window;       /* views, >= 0 */
    int32_t n_sink;       /* tokens, >= 0 */
    int32_t causal;
} saf3r_window;

/* Query and output rows of a step. */
typedef struct {
    int32_t n_heads;      /* query heads, 1..64, a multiple of the cache's heads: head h reads kv head h / (n_heads / kv heads) */
    int32_t out_is_fp32;
    const void* q;        /* bf16, n_tokens x n_heads rows of 64 */
    int64_t q_token_stride, q_head_stride;
    void* out;            /* bf16 or fp32; no row of it overlaps one of q, or the cache */
    int64_t out_token_stride, out_head_stride;
} saf3r_query_rows;

/* Workspace bytes of saf3r_kv_attn for these sizes (pointers are not read; 0 for invalid arguments). */
size_t saf3r_kv_attn_workspace_bytes(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch,
                                     const saf3r_window* window, int n_heads);

/*
 * Attention of each sequence's new tokens to its cached tokens, themselves among them (append first):
 * softmax(q . k / sqrt(64)) over the tokens that `window` lets them see.  Pages without a visible token are not
 * read: the caller may have given them to others.  Up to 64 rows per sequence and kv head (max_new * heads per kv head)
 * take a kernel that splits the keys over the GPU; more the tensor-core kernel.  The longest sequence of the step decides for
 * all of them: one long chunk among single tokens costs these a tile of 128 rows each.
 * Weights are rounded once: over bf16 caches to 16 bits for up to 64 rows and to bf16's 8 bits from 65 on (the error of a row
 * grows from the output's rounding, 0.0017 of it, to 0.0024); over 8-bit caches to fp16 (those below 2^-14 of a row's first
 * logits' largest weight lose bits, 2^-25 of it at most).  Over 8-bit caches a row's queries are fp16 relative to its largest
 * (what is below 2^-14 of that loses bits, 2^-25 of it at most).  The tensor-core kernel computes one exponential in eight by a
 * cubic (8.6e-5 of the weight).  Sums are in fp32.
 * What a masked token holds never reaches a row.  A row is computed key by key, in fp32 at 0.11 us a key (70 times as long as the
 * other rows of a view),
 *   - next to a masked token whose values are not finite, and where a value in sight is infinite (up to 64 rows over bf16
 *     caches: or NaN);
 *   - where its values are so large that sums of them leave fp32's range (from about 1e34 on);
 *   - over 8-bit caches where the value scales of its pages are far apart: more than 2^64 for up to 64 rows, else 2^22 (pages of
 *     zeros, of scale 2^-100, do not count); and, from 65 rows on, where the key scales are more than 2^22 apart and the row's
 *     largest query times the largest key exceeds about 2^15;
 *   - from 65 rows on over bf16 caches where later logits exceed the largest of the first 128 keys of the row (or of one of the
 *     parts that its keys are cut into) by 44 (a weight of 2^64).
 * A warp may have 32 such rows while others wait for it: over more than half a million keys raise saf3r_set_wait_budget, or
 * the call may end with SAF3R_ERR_TIMEOUT.
 * A row whose logits are all minus infinity, or of which one is plus infinity or NaN, is NaN.
 * workspace: DEVICE, 16-byte aligned, saf3r_kv_attn_workspace_bytes bytes, used by one call at a time
 * (also when calls are captured: graphs that share it must not overlap); it needs no start value.
 */
saf3r_status saf3r_kv_attn(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch, const saf3r_window* window,
                           const saf3r_query_rows* rows, void* workspace, void* stream);

/* Workspace bytes of saf3r_window_attn (0 for invalid arguments). */
size_t saf3r_window_attn_workspace_bytes(const saf3r_layout* layout, const saf3r_window* window);

/*
 * Attention over views held at once, q, k, v and out as saf3r_dense_attn, each token seeing what `window`
 * says (view_tokens is usually the layout's V, but need not be).  out overlaps none of the others.  Workspace, precision and
 * rows computed key by key as saf3r_kv_attn with more than 64 rows over a bf16 cache.
 */
saf3r_status saf3r_window_attn(const saf3r_layout* layout, const saf3r_window* window, const void* q, const void* k,
                               const void* v, void* out, int out_is_fp32, void* workspace, void* stream);

/*
 * Timing hook for measurement: when start and stop are both non-NULL
 * cudaEvent_t handles, every following saf3r_sparse_attn / saf3r_dense_attn
 * call made on this host thread records `start` on its stream right before
 * its attention kernel and `stop` right after it.  NULL, NULL switches the
 * hook off.  The events are owned by the caller.
 */
void saf3r_set_kernel_events(void* start, void* stop);

/*
 * Budget, in GPU clock cycles, of every bounded device wait (the attention
 * kernels' and the token-wise selection's pipeline waits) in the calls that
 * follow on this host thread; cycles <= 0 restores the default of 4e9 cycles
 * (about 2 s at 1.965 GHz).  When a wait runs out, its CTA records
 * SAF3R_ERR_TIMEOUT in the device error word, lets the copies it has in flight
 * land (a separate, fixed teardown budget), frees its tensor memory and exits;
 * the output rows of its unfinished work items are then left unwritten.
 */
void saf3r_set_wait_budget(long long cycles);

/*
 * Test hook for the timeout path.  The next saf3r_sparse_attn, saf3r_dense_attn,
 * saf3r_window_attn or (with its tensor-core kernel) saf3r_kv_attn call on this
 * host thread launches its attention kernel with
 * one softmax warp of the first CTA withholding its first "P is in tensor
 * memory" arrival, so the tensor-core warp's wait for it runs out after the wait
 * budget (see saf3r_set_wait_budget): nothing faults or hangs, every device wait
 * being bounded.  saf3r_check then returns SAF3R_ERR_TIMEOUT; the following
 * calls run normally.  Not for production use.
 */
void saf3r_test_withhold_arrive(void);

/*
 * Synchronize `stream`, then read and clear the calling device's error word.
 * Returns SAF3R_OK or the first device-side error recorded since the last check.
 */
saf3r_status saf3r_check(void* stream);

/* Number of kernels the last saf3r_* call on this host thread launched. */
int saf3r_last_launch_count(void);

/* Static text for a status code. */
const char* saf3r_status_string(saf3r_status status);

#ifdef __cplusplus
}
#endif

#endif /* SAF3R_H */
