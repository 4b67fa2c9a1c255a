/*
 * pred.h -- C ABI of the low-rank block predictor for a paged KV cache (MI355X / gfx950).
 *
 * What it computes (predictor.rs page, module doc): a seeded projection
 * P [head_dim, r] maps every query (Q @ P) and every key of a KV block (K @ P)
 * to rank r; the projected keys live in A_g [layers, max_blocks, num_kv_heads,
 * block_size, r] (bf16, layout comment on a_g_bytes and on the Predictor
 * fields); a block's score is the max, over query heads, query rows and the
 * block's tokens, of the projected dot product, and an ascending sort of the
 * scores ranks eviction victims (lowest score first).
 *
 * Conventions for every call below
 *   - Return value: 0 on success, a negative PRED_ERR_* code on failure; the
 *     thread-local pred_last_error() string then says what was wrong.  A call
 *     that fails argument checks enqueues nothing.
 *   - Pointers marked "device" are HIP device pointers the caller owns and
 *     keeps alive until the enqueued work has finished; "host" pointers are
 *     read or written before the call returns.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Every call except
 *     pred_create, pred_copy_projection, pred_read_slot and pred_device_error
 *     only enqueues work on `stream` and returns without synchronising
 *     (the pages' *_on_stream variants).
 *   - bf16 tensors are raw IEEE bfloat16 bit patterns (uint16_t), row-major.
 *   - The library allocates device memory only in pred_create (P, A_g and a
 *     4-byte error word) and frees it in pred_destroy.
 */
#ifndef PRED_H
#define PRED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t pred_bf16;
typedef struct pred_handle pred_t;

/* PredictorDims (predictor.rs page).  All fields must be > 0 and
 * num_q_heads must be a multiple of num_kv_heads (PredictorDims::validate). */
typedef struct {
    int32_t num_layers;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t r;
    int32_t block_size;
    int64_t max_blocks;
} pred_dims;

enum {
    PRED_OK = 0,
    PRED_ERR_INVALID_DIMS = -1, /* a dim <= 0, nq % nkv != 0, or a size overflows int64 */
    PRED_ERR_OUT_OF_RANGE = -2, /* layer / block / count outside the dims */
    PRED_ERR_OOM = -3,          /* A_g does not fit in 95% of free HBM */
    PRED_ERR_UNSUPPORTED = -4,  /* a shape this library's kernels do not handle */
    PRED_ERR_NULL_ARG = -5,     /* a required pointer is NULL */
    PRED_ERR_HIP = -6,          /* a HIP runtime call or kernel launch failed */
    PRED_ERR_WORKSPACE = -7,    /* workspace missing or too small */
    PRED_ERR_DEVICE = -8        /* a kernel met an invalid block-table entry */
};

/* pred_create flags */
#define PRED_FLAG_ZERO_AG 1u /* zero A_g after allocation (it is left unzeroed by default) */

/* ------------------------------------------------------------------ sizing (pure) */

/* Bytes of A_g: num_layers * max_blocks * num_kv_heads * block_size * r * 2
 * (predictor.rs page, a_g_bytes).  Returns a negative code if the dims are
 * invalid or the product overflows. */
int64_t pred_a_g_bytes(const pred_dims* d);

/* The fit check made by pred_create before it allocates A_g (predictor.rs
 * page, new_on_stream): A_g must not exceed 95% of `free_bytes`, the rest being
 * kept for scratch and attention.  Returns 0 if it fits, PRED_ERR_OOM with a
 * message naming r, max_blocks and the sizing formula otherwise, or
 * PRED_ERR_INVALID_DIMS.  No device access. */
int pred_check_fit(const pred_dims* d, uint64_t free_bytes);

/* Largest r and max_blocks this library's kernels accept, and other shape
 * limits, as a human-readable message (host string, static storage). */
const char* pred_limits(void);

/* ------------------------------------------------------------------ lifetime */

/* Validate the dims, build P on the host from `seed` (N(0, 1/r) rounded to
 * bf16 by the SplitMix64 / Box-Muller rule the library documents), check the
 * fit against hipMemGetInfo, allocate P and A_g on the current device, upload
 * P on `stream` and synchronise it (predictor.rs page, new_on_stream).
 * A_g is not zeroed unless PRED_FLAG_ZERO_AG is set: score_blocks may read
 * slots that project_kv_block never wrote.  On any failure everything
 * allocated is freed and *out is left NULL. */
int pred_create(const pred_dims* d, uint64_t seed, uint32_t flags, void* stream, pred_t** out);

/* As pred_create, but P is taken from `p_host` [head_dim, r] bf16 (host) instead
 * of being generated.  For tests that need a chosen P (identity, hand-worked
 * examples). */
int pred_create_with_projection(const pred_dims* d, const pred_bf16* p_host, uint32_t flags,
                                void* stream, pred_t** out);

/* Free P, A_g and the handle.  Waits for the device first.  NULL is a no-op. */
void pred_destroy(pred_t* p);

/* ------------------------------------------------------------------ hot path */

/* q_proj = bf16(q @ P) (predictor.rs page, project_q).
 *   q       device, [n_vec, num_q_heads, head_dim] bf16 (n_vec stacked query rows,
 *           e.g. layers x sequences x rows)
 *   q_proj  device, [n_vec, num_q_heads, r] bf16 output
 * Every output element is the float64 sum of its head_dim exact bf16 products,
 * rounded once to bf16 (nearest, ties to even).  n_vec == 0 is a no-op. */
int pred_project_q(pred_t* p, const pred_bf16* q, int64_t n_vec, pred_bf16* q_proj, void* stream);

/* Project whole KV blocks of `n_layers` layers and write their low-rank keys
 * into A_g through block tables (predictor.rs page, project_kv_block, batched
 * over blocks and layers).
 *   k            device, [n_layers, n_blocks, block_size, num_kv_heads, head_dim]
 *                bf16 (one block per [block_size, num_kv_heads, head_dim] slice,
 *                the page's k_block layout)
 *   block_table  device, [n_layers, n_blocks] int32 physical slot ids, or NULL
 *                for slots 0..n_blocks-1 in every layer
 * Block i of layer layer0 + l lands in A_g[layer0 + l, block_table[l, i]] as
 * [num_kv_heads, block_size, r], each element bf16(float64 sum).  Host-side
 * errors: layers outside [0, num_layers) or (NULL table) n_blocks > max_blocks
 * -> PRED_ERR_OUT_OF_RANGE.  A table entry outside [0, max_blocks) is skipped on
 * the device and raises the device error word (see pred_device_error).  Two
 * entries naming one slot of one layer race.  Any count of zero is a no-op. */
int pred_project_kv_block(pred_t* p, int32_t layer0, int32_t n_layers, const pred_bf16* k,
                          const int32_t* block_table, int64_t n_blocks, void* stream);

/* The two projections of one decode step in one call: exactly
 * pred_project_kv_block(p, layer0, n_layers, k_new, new_table, n_new, stream)
 * followed by pred_project_q(p, q, n_vec, q_proj, stream), with the same
 * arguments, checks and results (predictor.rs page: project_kv_block and
 * project_q, both run once per step).  Both parts are checked before either is
 * enqueued.  When both are small (a decode step's one new block per layer and
 * its query rows) they share one kernel launch, which saves a launch's fixed
 * cost on the step's critical path; larger calls take the two usual launches.
 *   k_new      device, [n_layers, n_new, block_size, num_kv_heads, head_dim] bf16
 *   new_table  device, [n_layers, n_new] int32 or NULL (slots 0..n_new-1)
 *   q          device, [n_vec, num_q_heads, head_dim] bf16
 *   q_proj     device, [n_vec, num_q_heads, r] bf16 output
 * A zero count skips its part. */
int pred_project_step(pred_t* p, int32_t layer0, int32_t n_layers, const pred_bf16* k_new,
                      const int32_t* new_table, int64_t n_new, const pred_bf16* q, int64_t n_vec,
                      pred_bf16* q_proj, void* stream);

/* Block scores (predictor.rs page, score_blocks, extended to several layers,
 * sequences and query rows).
 *   q_proj        device, [n_layers, n_seqs, n_rows, num_q_heads, r] bf16
 *   block_tables  device, [n_seqs, n_blocks] int32 physical ids, or NULL for the
 *                 identity (every sequence reads slots 0..n_blocks-1)
 *   scores        device, [n_layers, n_seqs, n_blocks] float32 output
 * scores[l, s, b] = max over rows i, query heads h, tokens t of
 *   sum_j q_proj[l, s, i, h, j] * A_g[layer0 + l, table[s, b], h / g, t, j]
 * with g = num_q_heads / num_kv_heads, accumulated in float32, no scale.
 * Scores are indexed by logical block position b.  Slots never written hold
 * whatever A_g held.  Errors: layer0 + n_layers > num_layers, n_blocks >
 * max_blocks with a NULL table -> PRED_ERR_OUT_OF_RANGE.  A table entry outside
 * [0, max_blocks) gives that block a NaN score and raises the device error word.
 * Any count of zero is a no-op. */
int pred_score_blocks(pred_t* p, int32_t layer0, int32_t n_layers, const pred_bf16* q_proj,
                      int32_t n_rows, const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs,
                      float* scores, void* stream);

/* As pred_score_blocks, but the last block of each sequence (logical block
 * n_blocks - 1) is partly filled: only its first last_fill[s] tokens are scored
 * (a decode step appends one token at a time; the predictor.rs page scores all
 * block_size tokens of every block, which equals last_fill[s] = block_size).
 *   last_fill  device, [n_seqs] int32 in [0, block_size], or NULL for full blocks.
 * A last block with fill 0 scores -inf.  A value outside [0, block_size] is
 * clamped to it and raises the device error word (see pred_device_error). */
int pred_score_blocks_masked(pred_t* p, int32_t layer0, int32_t n_layers, const pred_bf16* q_proj,
                             int32_t n_rows, const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs,
                             const int32_t* last_fill, float* scores, void* stream);

/* Eviction order (predictor.rs page, module doc: scores rank eviction victims;
 * qsa_select.rs page, host top-k: lower index on ties).
 *   scores     device, [n_segments, n_blocks] float32
 *   victims    device, [n_segments, n_blocks] int32 output: each row is the
 *              permutation of 0..n_blocks-1 that sorts the row's scores
 *              ascending, equal scores in ascending index order, -0 equal to
 *              +0, NaN before everything
 *   workspace  device scratch of at least pred_rank_workspace_bytes() bytes
 *              (may be NULL when that is 0)
 * n_blocks and n_segments must be <= 2^31 - 1.  A call too large for one
 * launch (over 2^31 - 1 workgroups) fails with PRED_ERR_OUT_OF_RANGE before
 * anything is enqueued; the same holds for the other entry points. */
int pred_rank_victims(pred_t* p, const float* scores, int64_t n_blocks, int64_t n_segments,
                      int32_t* victims, void* workspace, size_t ws_bytes, void* stream);

/* pred_rank_victims for callers that cannot allocate or pass a workspace:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments (without the workspace), checks and result as
 * pred_rank_victims; the sorted runs live instead in a static device array of
 * PRED_NOALLOC_SCRATCH_BYTES bytes that each GPU holds from library load to
 * process end (its address is found once per device by pred_create).  The call
 * allocates nothing and makes no memset: every byte of scratch it reads it has
 * written first in the same call.
 *   scores   device, [n_segments, n_blocks] float32
 *   victims  device, [n_segments, n_blocks] int32 output
 * A shape needing more than PRED_NOALLOC_SCRATCH_BYTES
 * (pred_rank_workspace_bytes(n_blocks, n_segments) above it, e.g. more than
 * 1048576 keys in rows of 2049..8192) fails with PRED_ERR_WORKSPACE before
 * anything is enqueued.  Every call on one GPU shares that GPU's array, across
 * handles and streams: two calls that can run at the same time on one GPU
 * (different streams or threads without ordering between them) race and give
 * wrong rankings; order them on one stream. */
#define PRED_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
int pred_rank_victims_noalloc(pred_t* p, const float* scores, int64_t n_blocks, int64_t n_segments,
                              int32_t* victims, void* stream);

/* The k lowest-scored blocks of every segment, in eviction order: row s of
 * victims is exactly the first k entries of pred_rank_victims's row s (scores
 * ascending, equal scores in ascending index order, -0 equal to +0, NaN
 * first).  This is the step after the ranking (predictor.rs page, module doc:
 * scores rank eviction victims; a cache evicts k blocks at a time).
 *   scores     device, [n_segments, n_blocks] float32
 *   k          0 <= k <= n_blocks (k = n_blocks is the full ranking)
 *   victims    device, [n_segments, k] int32 output (row stride k)
 *   workspace  as for pred_rank_victims (pred_rank_workspace_bytes(n_blocks,
 *              n_segments) bytes; NULL when that is 0)
 * Only each sorted run's first k places are merged, so small k costs less
 * than the full ranking. */
int pred_select_victims(pred_t* p, const float* scores, int64_t n_blocks, int64_t n_segments, int64_t k,
                        int32_t* victims, void* workspace, size_t ws_bytes, void* stream);

/* Name of the kernel pred_score_blocks (and pred_score_blocks_masked) runs for
 * this handle's dims and n_rows query rows per sequence (host only, static
 * string): "score_prefill_kernel" (more than 16 queries per kv head: bf16
 * MFMA), "score_decode_mfma_kernel" (5 to 16), "score_decode_kernel" (up to 4,
 * or shapes the matrix-core variant does not take) or "score_generic_kernel"
 * (r or block_size outside the streaming layouts).  NULL for a NULL handle or
 * n_rows < 1. */
const char* pred_score_kernel_name(pred_t* p, int32_t n_rows);

/* As pred_score_kernel_name, with the kernel's template arguments for a call
 * of n_blocks blocks per sequence, e.g.
 * "score_decode_kernel<lanes_per_row=4,queries=4,slots=2,q_in_lds=1,offset=u32,uniform_slots=1>"
 * (q_in_lds: the q_proj slab of one (layer, sequence) is staged in LDS, which
 * it is up to 32 KiB; offset: u64 when one layer of A_g is 4 GiB or more).
 * Host only; the string is thread-local storage valid until the next call on
 * the same thread.  NULL for a NULL handle, n_rows < 1 or n_blocks < 1. */
const char* pred_score_kernel_variant(pred_t* p, int32_t n_rows, int64_t n_blocks);

/* Score kernel override, a debugging switch (qsa_select.rs page: the prefill
 * selection's environment switch that forces its scalar scorer in place of the
 * tensor-core one).  PRED_SCORE_PATH_AUTO is the library's own choice; _DECODE
 * routes every pred_score_blocks / pred_score_blocks_masked call through the
 * vector-ALU streaming decode kernel (or the plain kernel where its layout does
 * not fit); _GENERIC routes those and pred_score_rows through the plain
 * per-block / per-cell kernels.  Every path gives the same scores within
 * float32 rounding.  The initial value comes from the environment variable
 * PRED_SCORE_PATH (auto, decode or generic), read once per process; the
 * variable PRED_LOG=1 makes every score launch print one line on stderr naming
 * its kernel.  Process-wide, not tied to a handle; set it while no other
 * thread is enqueueing score calls. */
enum { PRED_SCORE_PATH_AUTO = 0, PRED_SCORE_PATH_DECODE = 1, PRED_SCORE_PATH_GENERIC = 2 };
/* Returns 0, or PRED_ERR_OUT_OF_RANGE for a value not in the enum above. */
int pred_set_score_path(int32_t path);
/* The current PRED_SCORE_PATH_* value (host only, no device needed). */
int pred_get_score_path(void);

/* Per-row causal block scores of a prefill chunk (qsa_select.rs page, prefill
 * selection: each query row is scored against the blocks complete at its
 * position; the score is the predictor's, predictor.rs page, score_blocks, kept
 * per row instead of maximised over rows).
 *   layer        A_g layer to read, 0 <= layer < num_layers
 *   q_proj       device, [rows, num_q_heads, r] bf16; row i sits at position
 *                first_pos + i of the sequence
 *   block_table  device, [n_blocks] int32 physical ids of the sequence's
 *                blocks, or NULL for slots 0..n_blocks-1
 *   scores       device, [rows, stride] float32 output
 * With complete(i) = min(n_blocks, (first_pos + i + 1) / block_size), the
 * blocks whose every token is at or before row i's position:
 *   scores[i, b] = max over query heads h, tokens t of
 *                  sum_j q_proj[i, h, j] * A_g[layer, table[b], h / g, t, j]
 * for b < complete(i) (float32 accumulation, no scale), and -inf for
 * complete(i) <= b < stride.  A table entry outside [0, max_blocks) gives a
 * complete block a NaN score and raises the device error word.  rows and
 * n_blocks <= 2^31-1; rows * stride == 0 is a no-op; q_proj must be 16-byte
 * aligned. */
int pred_score_rows(pred_t* p, int32_t layer, const pred_bf16* q_proj, int64_t rows, int64_t first_pos,
                    const int32_t* block_table, int64_t n_blocks, float* scores, int64_t stride,
                    void* stream);

/* Per-row keep sets (qsa_select.rs page, prefill selection's top-k per row,
 * here on the device): for row i the first c(i) = min(stride,
 * (first_pos + i + 1) / ratio) entries of scores row i, ordered by descending
 * score with equal scores in ascending index order (-0 equal to +0, NaN after
 * everything), and the first topk of them written to keep row i.  Slots past
 * c(i) hold -1.
 *   scores     device, [rows, stride] float32 (e.g. pred_score_rows's output,
 *              with ratio = block_size)
 *   keep       device, [rows, topk] int32 output
 *   ratio      >= 1; first_pos in [0, 2^62]; 0 <= topk <= stride
 *   workspace  pred_rank_workspace_bytes(stride, rows) bytes (NULL when 0)
 * rows and stride must be <= 2^31-1. */
int pred_select_keep(pred_t* p, const float* scores, int64_t rows, int64_t stride, int64_t first_pos,
                     int32_t ratio, int64_t topk, int32_t* keep, void* workspace, size_t ws_bytes,
                     void* stream);

/* One decode step in one call: the step's new blocks into A_g, q_proj of every
 * layer, block scores and each (layer, sequence) row's k lowest blocks in
 * eviction order -- pred_project_step (pred_project_kv_block and
 * pred_project_q), pred_score_blocks_masked and pred_select_victims (pred_rank_victims when
 * k = n_blocks) on one stream, in that order, with the same arguments and
 * results (predictor.rs page: project_q, project_kv_block and score_blocks of
 * one step; module doc: the scores rank eviction victims).
 *   k_new       device, [n_layers, n_new, block_size, num_kv_heads, head_dim] bf16
 *   new_table   device, [n_layers, n_new] int32 slots for them (NULL: 0..n_new-1)
 *   q           device, [n_layers, n_seqs, n_rows, num_q_heads, head_dim] bf16
 *   q_proj      device, [n_layers, n_seqs, n_rows, num_q_heads, r] bf16 output
 *   block_tables, n_blocks, n_seqs, last_fill: as for pred_score_blocks_masked
 *   scores      device, [n_layers, n_seqs, n_blocks] float32 output
 *   victims     device, [n_layers * n_seqs, k] int32 output, 0 <= k <= n_blocks
 *   workspace   pred_rank_workspace_bytes(n_blocks, n_layers * n_seqs) bytes
 * Every part's arguments are checked before anything is enqueued.  The step
 * allocates nothing, never synchronises and issues no memset, so a caller may
 * capture it into a HIP graph and replay it (the arguments are then fixed). */
int pred_decode_step(pred_t* p, int32_t layer0, int32_t n_layers, const pred_bf16* k_new,
                     const int32_t* new_table, int64_t n_new, const pred_bf16* q, int32_t n_rows,
                     pred_bf16* q_proj, const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs,
                     const int32_t* last_fill, float* scores, int64_t k, int32_t* victims,
                     void* workspace, size_t ws_bytes, void* stream);

/* Workspace pred_rank_victims needs for this shape: 0 for n_blocks <= 2048
 * (each segment is sorted inside one workgroup), else 8 bytes per key for the
 * sorted runs, twice that for n_blocks > 8192 (pairwise merge buffers). */
size_t pred_rank_workspace_bytes(int64_t n_blocks, int64_t n_segments);

/* ------------------------------------------------------------------ the paged KV cache
 *
 * The operators around the predictor: putting new tokens into a paged KV cache
 * with rotary positions, attending over that cache, and evicting from it by the
 * attention its blocks really gathered -- the measured counterpart of the
 * predicted block score, ranked by the same rule.  A decode or verify step runs
 *   pred_rotate_store, pred_attend, (the caller accepts drafted tokens),
 *   pred_accumulate_weight, pred_evict_blocks
 * on one stream.  None of these calls allocates, synchronises or issues a
 * memset, so a caller may capture them into a HIP graph.  They take num_q_heads,
 * num_kv_heads, head_dim, block_size and max_blocks from the handle, and the
 * handle's device must be the current one (PRED_ERR_OUT_OF_RANGE otherwise). */

/* Element type of a KV cache: bf16; 8-bit e4m3 (1 sign, 4 exponent, 3 fraction
 * bits, no infinities, largest value 448); or 4-bit e2m1 (0, 0.5, 1, 1.5, 2, 3,
 * 4, 6 and their negatives) with one power of two for each 32 of a head's values,
 * 17/32 of a byte a value. */
enum { PRED_KV_BF16 = 0, PRED_KV_FP8 = 1, PRED_KV_FP4 = 2 };

/* One layer's paged KV cache, memory of the caller's.  Token t of block b, head
 * h is head_dim consecutive elements at
 *   b * block_stride + t * token_stride + h * head_stride
 * (strides in elements, the same for k and v), so both [max_blocks, block_size,
 * num_kv_heads, head_dim] (the layout pred_project_kv_block reads) and
 * [max_blocks, num_kv_heads, block_size, head_dim] (A_g's) are views of it.
 * k, v and every stride must be multiples of 16 bytes (bf16) or 8 bytes (FP8),
 * token_stride and head_stride >= head_dim, and block_stride at least one
 * block's extent.  An element stands for scale * stored; with bf16 and FP4 both
 * scales must be 1.
 *
 * FP4: head_dim and the strides are multiples of 32, k and v 16-byte aligned.
 * The element at offset x is the low (x even) or high nibble of byte x / 2, and
 * stands for its e2m1 value times 2^(b - 127), b the byte at offset x / 32 of
 * k_scales or v_scales; b = 255 makes its 32 values NaN; 0, 1, 253 and 254, whose
 * values bf16 does not all hold, are not written by the library and must not be
 * given.  So a cache [max_blocks,
 * block_size, num_kv_heads, head_dim / 2] of bytes has scales [.., head_dim / 32]
 * with the same order of dimensions.  The other types do not read k_scales and
 * v_scales. */
typedef struct {
    void* k;
    void* v;
    int64_t block_stride, token_stride, head_stride;
    int32_t dtype;
    float k_scale, v_scale;
    uint8_t* k_scales;
    uint8_t* v_scales;
} pred_kv_cache;

/* How a rotation's frequencies are stretched for contexts longer than the model
 * was trained on (pred_rope_scaling.kind). */
enum {
    PRED_ROPE_NONE = 0,   /* f_i = theta^(-2 i / rot_dim) */
    PRED_ROPE_LINEAR = 1, /* f_i / factor */
    PRED_ROPE_NTK = 2,    /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta */
    PRED_ROPE_LLAMA3 = 3, /* f_i where its wavelength 2 pi / f_i is below original_length / high, f_i / factor
                             where it is above original_length / low, and between them
                             (1 - m) f_i / factor + m f_i, m = (original_length / wavelength - low) / (high - low) */
    PRED_ROPE_YARN = 4    /* f_i / factor * ramp_i + f_i * (1 - ramp_i), ramp_i = clamp((i - a) / max(b - a, 0.001),
                             0, 1), a = max(floor(d(high)), 0), b = min(ceil(d(low)), rot_dim - 1), d(n) = rot_dim *
                             ln(original_length / (2 pi n)) / (2 ln theta); mscale = 0.1 ln(factor) + 1 */
};
typedef struct {
    int32_t kind;
    double factor, low, high, original_length;
} pred_rope_scaling;

/* A rotation: `turns` is the device copy of pred_rope_turns's output. */
typedef struct {
    const uint64_t* turns; /* device, [rot_dim / 2] */
    int32_t rot_dim;       /* the first rot_dim values of a head turn, the others pass; even, <= head_dim */
    int32_t interleaved;   /* pairs (2 i, 2 i + 1) if not 0, else (i, i + rot_dim / 2) */
    int32_t backward;      /* not 0: the transposed map, the gradient of the rotation */
    float mscale;          /* factor on cosine and sine */
} pred_rope;

/* Frequencies of a rotation, on the host (no device access): turns[i] is
 * f_i / (2 pi), the turns a position adds to pair i, as a 64-bit binary
 * fraction (value * 2^64, modulo whole turns).  position * turns[i] modulo 2^64
 * is then the angle of any position without loss: its error is under
 * |position| * 2^-53 turns, where a float32 angle would be off by radians.
 * `scaling` NULL means PRED_ROPE_NONE.  mscale (host, may be NULL) receives the
 * factor for pred_rope.mscale.  PRED_ERR_OUT_OF_RANGE for rot_dim odd, < 2 or
 * > 65536, theta <= 1, a factor <= 0, an unknown kind, rot_dim 2 with NTK, or
 * low, high, original_length that the kind cannot use (LLAMA3: 0 < low < high
 * and original_length > 0; YARN: low, high and original_length > 0). */
int pred_rope_turns(int32_t rot_dim, double theta, const pred_rope_scaling* scaling, uint64_t* turns, float* mscale);

/* Rotary positions: for token t, head h and pair (a, b) at frequency f,
 *   out_a = mscale * (x_a cos(pos f) - x_b sin(pos f))
 *   out_b = mscale * (x_a sin(pos f) + x_b cos(pos f))
 * (rope->backward: sin negated -- the gradient with respect to x of a forward
 * call, given the gradient of its output), computed in float32 and rounded once
 * to bf16.  Values past rot_dim are copied.
 *   x          device, [n_tokens, n_heads, head_dim] bf16, tokens x_stride elements apart
 *   positions  device, [n_tokens] int32 (any value, negative ones turn back)
 *   out        device, as x with out_stride; may be x itself (same stride), else it must not overlap it
 * x, out and the strides must be multiples of 16 bytes, strides >= n_heads *
 * head_dim; head_dim <= 512 (PRED_ERR_UNSUPPORTED above). */
int pred_rotate(pred_t* p, const pred_rope* rope, const pred_bf16* x, int64_t x_stride, int64_t n_tokens,
                int32_t n_heads, const int32_t* positions, pred_bf16* out, int64_t out_stride, void* stream);

/* The start of a step over the cache, in one launch: the new tokens' queries and
 * keys rotated as by pred_rotate, the queries to q_out, the keys and the values
 * into the cache.
 *   q, k, v    device, [n_tokens, num_q_heads | num_kv_heads | num_kv_heads, head_dim] bf16, tokens q_stride,
 *              k_stride, v_stride elements apart (so all three may lie side by side in one buffer)
 *   slots      device, [n_tokens] int64: where a token goes, block * block_size + offset; -1 stores nothing
 *              (a padding token).  Any other value outside the cache stores nothing and raises the device error
 *              word.  Two tokens with one slot race.
 *   q_out      device, [n_tokens, num_q_heads, head_dim] bf16; may be q itself if q_stride is num_q_heads * head_dim
 * A bf16 cache takes keys and values rounded once; an FP8 cache takes value /
 * scale, a float32 quotient, clamped to +-448 and rounded to the nearest (ties to
 * even), NaN kept.  An FP4 cache takes values rounded to bf16: the scale of 32 is
 * the smallest power of two, at least 2^-125 and at most 2^125, that keeps the
 * largest of them within 6, each value then the nearest (ties to the even
 * pattern); a value that is not finite makes its 32 values NaN.
 * rope->backward must be 0, and the cache's k and v must not overlap (one
 * address for both is PRED_ERR_OUT_OF_RANGE). */
int pred_rotate_store(pred_t* p, const pred_rope* rope, const pred_bf16* q, int64_t q_stride, const pred_bf16* k,
                      int64_t k_stride, const pred_bf16* v, int64_t v_stride, int64_t n_tokens,
                      const int32_t* positions, const int64_t* slots, const pred_kv_cache* cache, pred_bf16* q_out,
                      void* stream);

/* A norm of a head's values, as models put on queries and keys before the rotation:
 *   x -> x / sqrt(mean(x^2) + eps) * (offset + weight)
 * over the head_dim values of each head, in float32 (a sum of squares above
 * float32's range gives 0 or NaN).  weight: device, [head_dim] bf16, 16-byte aligned, or NULL
 * for a factor of 1 (offset then counts for nothing).  eps > 0. */
typedef struct {
    const pred_bf16* weight;
    float eps;
    float offset;
} pred_norm;

/* pred_rotate with a norm before it, in one pass: out = R(pos) norm(x), rounded
 * once.  rope NULL: the norm alone (positions may be NULL); rope->backward must
 * be 0.  The other arguments and their limits are pred_rotate's; out may be x
 * itself. */
int pred_norm_rotate(pred_t* p, const pred_norm* norm, const pred_rope* rope, const pred_bf16* x, int64_t x_stride,
                     int64_t n_tokens, int32_t n_heads, const int32_t* positions, pred_bf16* out, int64_t out_stride,
                     void* stream);

/* Its gradient: from x as it went in and dy, the gradient of out (bf16, tokens
 * dy_stride apart),
 *   dx       bf16, tokens dx_stride apart; may be x or dy itself (same stride), else it must not overlap them
 *   dweight  device, [head_dim] float32 or NULL: the gradient of (offset + weight), summed over tokens and heads in
 *            float32 in a fixed order (equal inputs give equal bits); written, not added to
 *   workspace  pred_norm_rotate_workspace_bytes() bytes, 16-byte aligned; NULL without dweight
 * With dweight a second launch adds the workgroups' sums. */
int pred_norm_rotate_backward(pred_t* p, const pred_norm* norm, const pred_rope* rope, const pred_bf16* x,
                              int64_t x_stride, int64_t n_tokens, int32_t n_heads, const int32_t* positions,
                              const pred_bf16* dy, int64_t dy_stride, pred_bf16* dx, int64_t dx_stride, float* dweight,
                              void* workspace, size_t ws_bytes, void* stream);

/* Workspace of pred_norm_rotate_backward with dweight, at most 1024 * head_dim
 * bytes; 0 for a NULL handle or counts < 1.  Calls that may run at the same time
 * need workspaces of their own. */
size_t pred_norm_rotate_workspace_bytes(pred_t* p, int64_t n_tokens, int32_t n_heads);

/* pred_rotate_store with norms before the rotation, in the same launch: q_norm on
 * the queries, k_norm on the keys, either NULL for none; rope NULL for no
 * rotation (positions may be NULL then). */
int pred_norm_rotate_store(pred_t* p, const pred_norm* q_norm, const pred_norm* k_norm, const pred_rope* rope,
                           const pred_bf16* q, int64_t q_stride, const pred_bf16* k, int64_t k_stride,
                           const pred_bf16* v, int64_t v_stride, int64_t n_tokens, const int32_t* positions,
                           const int64_t* slots, const pred_kv_cache* cache, pred_bf16* q_out, void* stream);

/* Keys and values into the cache as they are (already rotated, or of a layer
 * without rotation), rounded as by pred_rotate_store; k, v and slots as there. */
int pred_store(pred_t* p, const pred_bf16* k, int64_t k_stride, const pred_bf16* v, int64_t v_stride, int64_t n_tokens,
               const int64_t* slots, const pred_kv_cache* cache, void* stream);

/* Cached tokens read back: what the elements at `slots` (as for pred_rotate_store)
 * stand for, rounded to bf16 (exact for bf16 and FP4 caches), into k_out and
 * v_out, device, [n_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned.  A
 * token whose slot is -1 or outside the cache leaves its rows as they were; the
 * latter raises the device error word.  k_out and v_out must not overlap
 * (PRED_ERR_OUT_OF_RANGE); num_kv_heads * head_dim <= 2^30 (PRED_ERR_UNSUPPORTED). */
int pred_load(pred_t* p, const pred_kv_cache* cache, int64_t n_tokens, const int64_t* slots, pred_bf16* k_out,
              pred_bf16* v_out, void* stream);

/* Attention of each sequence's newest tokens over its cached ones: one token
 * (n_rows = 1, a decode step) or a tree of drafted tokens to verify.  A
 * sequence's tokens 0 .. kv_len - 1 lie in the blocks of its table in order, the
 * drafted ones last; with d = draft_len, row i < d is token kv_len - d + i.  It
 * sees every token before kv_len - d (the context), and drafted token j if bit j
 * of its tree word is set.
 *   q             device, [n_seqs, n_rows, num_q_heads, head_dim] bf16, 1 <= n_rows <= 64
 *   tree          device, [n_seqs, n_rows] 64-bit words, or NULL for a chain (row i sees drafted tokens 0 .. i)
 *   block_tables  device, [n_seqs, n_blocks] int32 physical ids, or NULL for the identity
 *   kv_len        device, [n_seqs] int32 in [0, n_blocks * block_size], or NULL for that upper limit
 *   draft_len     device, [n_seqs] int32 in [0, min(n_rows, kv_len)], or NULL for that upper limit
 *   out           device, [n_seqs, n_rows, num_q_heads, head_dim] bf16: softmax(scale * q k) v over the row's tokens;
 *                 must not overlap q (PRED_ERR_OUT_OF_RANGE)
 *   lse           device, [n_seqs, n_rows, num_q_heads] float32 or NULL: the log of the softmax's sum
 *   block_lse     device, [n_seqs, n_blocks, n_rows, num_q_heads] float32 or NULL: the same sum over each block's
 *                 tokens alone, for pred_accumulate_weight; blocks at or past kv_len / block_size rounded up are left
 *                 as they were
 *   workspace     device scratch of pred_attend_workspace_bytes() bytes, 16-byte aligned (NULL when that is 0)
 * A row past draft_len and a row that sees no token have output 0 and lse -inf.
 * Query head h reads kv head h / (num_q_heads / num_kv_heads).  Scores, sums and
 * the softmax are held in float32; in the stream and tree kernels a weight enters
 * its product with a value as two bf16 terms, 16 of its bits.  What a masked token
 * holds (NaN, infinities) does not reach a row that cannot see it.  An infinite
 * value that a row sees makes that element of its output the infinity, however
 * small its weight; NaN, and infinities of both signs, make it NaN.  Lengths
 * outside their range are clamped, and a block whose table entry is outside [0,
 * max_blocks) is left out of every sum; both raise the device error word.
 * head_dim <= 256 (PRED_ERR_UNSUPPORTED above); n_blocks * block_size <= 2^29
 * (here and in the two calls below). */
int pred_attend(pred_t* p, const pred_kv_cache* cache, const pred_bf16* q, int32_t n_rows, const uint64_t* tree,
                const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs, const int32_t* kv_len,
                const int32_t* draft_len, float scale, pred_bf16* out, float* lse, float* block_lse, void* workspace,
                size_t ws_bytes, void* stream);

/* Workspace of pred_attend for this shape on this handle (partial results of a
 * long context split over workgroups); 0 for a NULL handle or counts < 1.  Calls
 * that may run at the same time need workspaces of their own.  It grows with the
 * queries per kv head and hardly with the context: on 256 CUs 1 MiB for one
 * sequence of 131072 tokens, 9 MiB for 64 sequences of one row (32 query and 8 kv
 * heads of 128), 292 MiB for 16 sequences of 64 rows (64 and 8 heads). */
size_t pred_attend_workspace_bytes(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks);

/* Name of the kernel pred_attend runs for this handle, cache and shape (host
 * only, static string), for head sizes 64 and 128: "attend_stream_kernel" (up to
 * 32 queries per kv head, block sizes a multiple of 1024 / (head_dim * element
 * bytes), a block's tokens within 2 GiB) or "attend_tree_kernel" (the others).
 * "attend_plain_kernel" for other head sizes, cache rows off 16-byte alignment,
 * and block_lse with a block size other than 8, 16 or a multiple of 32 up to
 * 65536.  NULL for a NULL argument, and for n_rows, a cache or a head size that
 * pred_attend refuses. */
const char* pred_attend_kernel_name(pred_t* p, const pred_kv_cache* cache, int32_t n_rows, int32_t with_block_lse);

/* Attention of each sequence's newest tokens with a sliding window: any number
 * of rows (a decode step's, a chain of drafted tokens, a prompt chunk, a whole
 * prompt).  With d = row_len, row i < d is token p = kv_len - d + i and sees the
 * `window` newest tokens up to itself, p - window + 1 .. p, and the sequence's first
 * n_sinks up to itself; window INT32_MAX hides nothing.
 *   n_rows    [1, 2^24], at most 2^30 queries per kv head; where a row sees up to 8192 tokens the work is divided by
 *             it, so a call of few rows is best made with few n_rows (16 rows, window 4096: 27 us, of 2048 99)
 *   row_len   device, [n_seqs] int32 in [0, min(n_rows, kv_len)], or NULL for that upper limit
 *   window    >= 1;  n_sinks >= 0
 * The other arguments, and what is said of rows past row_len, of masked tokens,
 * of values that are not finite and of lengths and entries out of range, are
 * pred_attend's.  Entries of blocks of which no row sees a token need not be
 * valid: those blocks may have been given back.  A weight enters its product with a
 * value as in pred_attend up to 16 queries per kv head (n_rows * num_q_heads /
 * num_kv_heads); above that, in the chunk kernel, as one bf16 term, so an output is
 * off by up to 2^-8 of the weighted mean of the absolute values more. */
int pred_attend_window(pred_t* p, const pred_kv_cache* cache, const pred_bf16* q, int32_t n_rows,
                       const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs, const int32_t* kv_len,
                       const int32_t* row_len, int32_t window, int32_t n_sinks, float scale, pred_bf16* out, float* lse,
                       void* workspace, size_t ws_bytes, void* stream);

/* Workspace of pred_attend_window for this shape on this handle; 0 for a NULL
 * handle or arguments that the call refuses, and where no walk is split: short
 * windows, and prompts of many rows that see up to 8192 tokens.  Calls that may run
 * at the same time need workspaces of their own.  On 256 CUs one sequence needs at
 * most 57 MiB.  Of several of which a row may see more than 8192 tokens it grows
 * with n_seqs * n_rows, by 4 * (head_dim + 2) bytes for each query: 413 MiB for two
 * prompts of 12000 rows (32 query and 8 kv heads of 128), 3.1 GiB for two of 100000. */
size_t pred_attend_window_workspace_bytes(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks, int32_t window,
                                          int32_t n_sinks);

/* As pred_attend_kernel_name: "attend_stream_kernel" (up to 16 queries per kv
 * head, the caches it takes there), "attend_chunk_kernel" (the others, head sizes
 * 64 and 128) or "attend_plain_kernel". */
const char* pred_attend_window_kernel_name(pred_t* p, const pred_kv_cache* cache, int32_t n_rows);

/* Accumulated attention weight of each block, from pred_attend's lse and
 * block_lse:
 *   mass_out[s, b] = decay * mass[s, b] + sum over accepted rows i, heads h of
 *                    exp(block_lse[s, b, i, h] - lse[s, i, h])
 * for the blocks that kv_len tokens use; the others keep their mass.  Rows with
 * lse = -inf add nothing.
 *   accepted   device, [n_seqs] 64-bit words, bit i = row i counts (a draft's accepted tokens), or NULL for all
 *   kv_len     as for pred_attend
 *   mass       device, [n_seqs, n_blocks] float32
 *   mass_out   device, as mass; may be mass itself, else it must not overlap it
 * The order of the sum is fixed: equal inputs give equal bits. */
int pred_accumulate_weight(pred_t* p, const float* lse, const float* block_lse, int32_t n_rows,
                           const uint64_t* accepted, const int32_t* kv_len, int64_t n_blocks, int32_t n_seqs,
                           float decay, const float* mass, float* mass_out, void* stream);

/* Eviction to a budget of blocks.  A sequence uses n = kv_len / block_size
 * rounded up blocks; if that is above `budget`, the n - budget blocks of lowest
 * mass among blocks protect_first .. n - protect_last - 1 are evicted (all of
 * those if they are fewer), in pred_rank_victims's order: equal mass by lower
 * index first, -0 equal to +0, NaN lowest.
 *   tables_out   the kept blocks' entries in their order, then the evicted ones' in theirs; entries from n on as in
 *                block_tables.  So the evicted slots are the next ones the sequence fills, or a list to give back.
 *   mass_out     the kept blocks' mass in that order, then 0 for the evicted ones; from n on as in mass
 *   kv_len_out   kv_len - evicted * block_size
 *   evicted      [n_seqs] int32 output: the number of blocks evicted
 * block_tables, tables_out [n_seqs, n_blocks] int32; mass, mass_out [n_seqs,
 * n_blocks] float32; kv_len, kv_len_out [n_seqs] int32, kv_len never NULL.
 * Each output may be its input itself, else it must not overlap it.  budget >=
 * 0, protect_first >= 0, protect_last >= 1 (the last block, which may be partly
 * filled, stays; protect as many as hold drafted tokens).  Any [n_seqs,
 * n_blocks] float32 score works as mass, pred_score_blocks's among them.  A
 * kv_len outside [0, n_blocks * block_size] is clamped and raises the device
 * error word.
 *   workspace   pred_evict_workspace_bytes() bytes, 8-byte aligned (NULL when 0) */
int pred_evict_blocks(pred_t* p, const int32_t* block_tables, const float* mass, const int32_t* kv_len,
                      int64_t n_blocks, int32_t n_seqs, int64_t budget, int32_t protect_first, int32_t protect_last,
                      int32_t* tables_out, float* mass_out, int32_t* kv_len_out, int32_t* evicted, void* workspace,
                      size_t ws_bytes, void* stream);

/* Workspace of pred_evict_blocks: 0 for n_blocks <= 32768 (a sequence's entries
 * are held in registers), else 8 bytes per entry. */
size_t pred_evict_workspace_bytes(int64_t n_blocks, int32_t n_seqs);

/* ------------------------------------------------------------------ inspection */

/* The P that pred_create builds for (head_dim, r, seed), computed on the host
 * only (no device needed): `out` is [head_dim, r] bf16.  Returns
 * PRED_ERR_INVALID_DIMS for non-positive sizes. */
int pred_projection_host(int32_t head_dim, int32_t r, uint64_t seed, pred_bf16* out);

/* Copy P [head_dim, r] bf16 to `host_out` (synchronous). */
int pred_copy_projection(pred_t* p, pred_bf16* host_out);

/* Device address of A_g [num_layers, max_blocks, num_kv_heads, block_size, r]
 * bf16 (predictor.rs page, a_g_dev_ptr).  The library owns it. */
void* pred_a_g_ptr(pred_t* p);

/* Copy the A_g slot (layer, block) [num_kv_heads, block_size, r] bf16 to
 * `host_out` and synchronise `stream` (predictor.rs page, read_k_lr_slot). */
int pred_read_slot(pred_t* p, int32_t layer, int64_t block, pred_bf16* host_out, void* stream);

/* The dims the handle was created with (predictor.rs page, dims). */
int pred_get_dims(pred_t* p, pred_dims* out);

/* Synchronise `stream`, read and clear the device error word.  Returns 0, or
 * PRED_ERR_DEVICE if a kernel since the last call met an invalid table entry,
 * a last-block fill count outside [0, block_size], a cache slot outside the
 * cache or a sequence length outside its range. */
int pred_device_error(pred_t* p, void* stream);

/* Message for the last failing call on this thread ("" if none). */
const char* pred_last_error(void);

/* Library version string. */
const char* pred_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PRED_H */
