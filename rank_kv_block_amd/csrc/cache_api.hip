// C entry points of the paged KV cache operators: argument checks and dispatch.
#include <cmath>

#include "common.h"
#include "handle.h"
#include "kernels.h"
#include "pred.h"

using pred::fail;
using pred::hip_fail;
using pred::mul_ok;
using pred::ok;

namespace {

// The handle, and that its device is the current one (a launch goes to the
// current device, and the error word is the handle's).
int check_handle(pred_t* p, const char* what) {
    if (!p) return fail(PRED_ERR_NULL_ARG, "predictor is NULL");
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (dev != p->device)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: the handle lives on device %d, the current device is %d", what,
                    p->device, dev);
    return PRED_OK;
}

int check_cache(pred_t* p, const pred_kv_cache* c, pred::CacheView* out, const char* what) {
    if (!c || !c->k || !c->v) return fail(PRED_ERR_NULL_ARG, "%s: cache, its k or its v is NULL", what);
    if (c->dtype != PRED_KV_BF16 && c->dtype != PRED_KV_FP8 && c->dtype != PRED_KV_FP4)
        return fail(PRED_ERR_UNSUPPORTED, "%s: cache dtype %d is not PRED_KV_BF16, PRED_KV_FP8 or PRED_KV_FP4", what,
                    c->dtype);
    const pred_dims& d = p->d;
    const bool fp4 = c->dtype == PRED_KV_FP4;
    if (fp4 && (!c->k_scales || !c->v_scales))
        return fail(PRED_ERR_NULL_ARG, "%s: a 4-bit cache's k_scales or v_scales is NULL", what);
    if (fp4 && d.head_dim % 32 != 0)
        return fail(PRED_ERR_UNSUPPORTED, "%s: a 4-bit cache needs a head_dim (%d) that is a multiple of 32", what,
                    d.head_dim);
    if (fp4 && ((c->block_stride | c->token_stride | c->head_stride) & 31 || !pred::aligned16(c->k) ||
                !pred::aligned16(c->v)))
        return fail(PRED_ERR_UNSUPPORTED, "%s: a 4-bit cache's strides (%lld, %lld, %lld) must be multiples of 32 "
                    "elements and its k, v 16-byte aligned", what, (long long)c->block_stride,
                    (long long)c->token_stride, (long long)c->head_stride);
    const int64_t bs = c->block_stride, ts = c->token_stride, hs = c->head_stride;
    if ((bs | ts | hs) & 7 || !pred::aligned_to(c->k, c->dtype == PRED_KV_FP8 ? 8 : 16) ||
        !pred::aligned_to(c->v, c->dtype == PRED_KV_FP8 ? 8 : 16))
        return fail(PRED_ERR_UNSUPPORTED, "%s: cache strides (%lld, %lld, %lld) must be multiples of 8 elements and k, "
                    "v aligned to 8 elements", what, (long long)bs, (long long)ts, (long long)hs);
    // tokens of a block apart, heads apart, and a block's extent inside its stride: no two elements share a place
    int64_t te, he, extent;
    if (ts < d.head_dim || hs < d.head_dim || !mul_ok(d.block_size - 1, ts, &te) ||
        !mul_ok(d.num_kv_heads - 1, hs, &he) || te > INT64_MAX / 4 || he > INT64_MAX / 4 ||
        bs < te + he + d.head_dim || !mul_ok(d.max_blocks, bs, &extent) || extent > INT64_MAX / 4)
        return fail(PRED_ERR_OUT_OF_RANGE,
                    "%s: cache strides (block %lld, token %lld, head %lld) overlap: tokens and heads must be at least "
                    "head_dim (%d) apart and a block's stride cover its tokens and heads", what, (long long)bs,
                    (long long)ts, (long long)hs, d.head_dim);
    // one of the two inner strides must step over the whole of the other's extent
    if (d.block_size > 1 && d.num_kv_heads > 1 && ts < he + d.head_dim && hs < te + d.head_dim)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: cache token stride %lld and head stride %lld make tokens and heads "
                    "overlap", what, (long long)ts, (long long)hs);
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || std::isinf(c->k_scale) || std::isinf(c->v_scale))
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: cache scales must be positive and finite", what);
    if (c->dtype != PRED_KV_FP8 && (c->k_scale != 1.f || c->v_scale != 1.f))
        return fail(PRED_ERR_UNSUPPORTED, "%s: a bf16 or 4-bit cache has k_scale and v_scale of 1", what);
    *out = pred::CacheView{c->k, c->v, bs, ts, hs, c->dtype == PRED_KV_FP8, c->k_scale, c->v_scale, fp4,
                           fp4 ? c->k_scales : nullptr, fp4 ? c->v_scales : nullptr};
    return PRED_OK;
}

int check_rope(pred_t* p, const pred_rope* r, const char* what) {
    if (!r || !r->turns) return fail(PRED_ERR_NULL_ARG, "%s: rope or its turns is NULL", what);
    if (r->rot_dim < 2 || (r->rot_dim & 1) || r->rot_dim > p->d.head_dim)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: rot_dim (%d) must be even and in [2, head_dim = %d]", what, r->rot_dim,
                    p->d.head_dim);
    if (!std::isfinite(r->mscale)) return fail(PRED_ERR_OUT_OF_RANGE, "%s: mscale must be finite", what);
    if (!pred::aligned_to(r->turns, 8)) return fail(PRED_ERR_UNSUPPORTED, "%s: turns must be 8-byte aligned", what);
    if (p->d.head_dim > 512) return fail(PRED_ERR_UNSUPPORTED, "%s: head_dim (%d) above 512", what, p->d.head_dim);
    return PRED_OK;
}

// A bf16 tensor [n_tokens, heads, head_dim] with its tokens `stride` apart.
int check_rows(pred_t* p, const void* x, int64_t stride, int64_t heads, const char* what, const char* name) {
    if (!x) return fail(PRED_ERR_NULL_ARG, "%s: %s is NULL", what, name);
    if (!pred::aligned16(x) || (stride & 7))
        return fail(PRED_ERR_UNSUPPORTED, "%s: %s must be 16-byte aligned and its stride a multiple of 8", what, name);
    if (stride < heads * p->d.head_dim)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: %s's stride (%lld) is below one token's %lld elements", what, name,
                    (long long)stride, (long long)(heads * p->d.head_dim));
    return PRED_OK;
}

// r NULL: nothing turns.
pred::RopeArgs rope_args(pred_t* p, const pred_rope* r, const int32_t* positions, int64_t n_tokens) {
    pred::RopeArgs a{};
    if (r) {
        a.turns = r->turns;
        a.rot = r->rot_dim;
        a.interleaved = r->interleaved != 0;
        a.backward = r->backward != 0;
        a.mscale = r->mscale;
        a.positions = positions;
    }
    a.n_tokens = n_tokens;
    a.D = p->d.head_dim;
    a.N = p->d.max_blocks;
    a.B = p->d.block_size;
    a.err = p->err_dev;
    return a;
}

// A cache that a call writes: k and v, and their scales, at places of their own.
int check_store(const pred_kv_cache* c, const char* what) {
    if (c->k == c->v) return fail(PRED_ERR_OUT_OF_RANGE, "%s: the cache's k and v are one", what);
    if (c->dtype == PRED_KV_FP4 && c->k_scales == c->v_scales)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: the cache's k_scales and v_scales are one", what);
    return PRED_OK;
}

// n NULL: no norm.
int check_norm(pred_t* p, const pred_norm* n, pred::HeadNorm* out, const char* what) {
    *out = pred::HeadNorm{};
    if (p->d.head_dim > 512) return fail(PRED_ERR_UNSUPPORTED, "%s: head_dim (%d) above 512", what, p->d.head_dim);
    if (!n) return PRED_OK;
    if (!(n->eps > 0.f) || std::isinf(n->eps) || !std::isfinite(n->offset))
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: a norm's eps must be above 0 and finite, its offset finite", what);
    if (!pred::aligned16(n->weight))
        return fail(PRED_ERR_UNSUPPORTED, "%s: a norm's weight must be 16-byte aligned", what);
    *out = pred::HeadNorm{n->weight, 1, n->eps, n->offset};
    return PRED_OK;
}

// A rotation of the calls that may do without (NULL) and run forwards only.
int check_forward_rope(pred_t* p, const pred_rope* r, const char* what) {
    if (!r) return PRED_OK;
    const int rc = check_rope(p, r, what);
    if (rc == 0 && r->backward) return fail(PRED_ERR_UNSUPPORTED, "%s: rope->backward must be 0", what);
    return rc;
}

// Tokens of a sequence: with 2^29 no sum of lengths, runs and tiles passes 32 bits.
constexpr int64_t kMostTokens = 1ll << 29;

// Head sizes that pred_attend has a kernel for.
constexpr int kMostHead = 256;

// The table's extent and the counts shared by the calls over sequences.
int check_counts(pred_t* p, int64_t n_blocks, int32_t n_seqs, const char* what) {
    if (n_blocks < 0 || n_seqs < 0)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: negative count (n_blocks %lld, n_seqs %d)", what, (long long)n_blocks,
                    n_seqs);
    int64_t tokens;
    if (!mul_ok(n_blocks, p->d.block_size, &tokens) || tokens > kMostTokens)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: %lld blocks of %d tokens are above 2^29 tokens", what,
                    (long long)n_blocks, p->d.block_size);
    return PRED_OK;
}

int check_n_rows(int32_t n_rows, const char* what) {
    if (n_rows < 1) return fail(PRED_ERR_OUT_OF_RANGE, "%s: n_rows (%d) must be >= 1", what, n_rows);
    if (n_rows > 64) return fail(PRED_ERR_UNSUPPORTED, "%s: n_rows (%d) above 64 (one word of bits a row)", what, n_rows);
    return PRED_OK;
}

pred::AttendArgs attend_shape(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks) {
    pred::AttendArgs a{};
    a.N = p->d.max_blocks;
    a.n = (int)n_blocks;
    a.S = n_seqs;
    a.M = n_rows;
    a.Hq = p->d.num_q_heads;
    a.Hk = p->d.num_kv_heads;
    a.D = p->d.head_dim;
    a.B = p->d.block_size;
    a.n_cu = p->n_cu;
    a.err = p->err_dev;
    return a;
}

bool attend_counts_ok(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks) {
    return n_seqs >= 1 && n_rows >= 1 && n_rows <= 64 && n_blocks >= 1 &&
           n_blocks <= kMostTokens / p->d.block_size;
}

// Rows of a sequence in a call with a window: up to 2^24, and up to 2^30 queries of a kv head.
bool window_rows_ok(pred_t* p, int32_t n_rows) {
    return n_rows >= 1 && n_rows <= 1 << 24 && (int64_t)n_rows * (p->d.num_q_heads / p->d.num_kv_heads) <= 1 << 30;
}

int check_window(pred_t* p, int32_t n_rows, int32_t window, int32_t n_sinks, const char* what) {
    if (!window_rows_ok(p, n_rows))
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: n_rows (%d) outside [1, 2^24], or more than 2^30 queries per kv head", what,
                    n_rows);
    if (window < 1 || n_sinks < 0)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: window (%d) must be >= 1 and n_sinks (%d) >= 0", what, window, n_sinks);
    return PRED_OK;
}

// No sequence has more than kMostTokens, so a larger window or more sinks hide nothing either.
void set_window(pred::AttendArgs* a, int32_t window, int32_t n_sinks) {
    a->window = window < kMostTokens ? window : (int)kMostTokens;
    a->sinks = n_sinks < kMostTokens ? n_sinks : (int)kMostTokens;
}

// The checks and the launch of both attention calls; `a` holds the shape and what
// only one of them has.
int attend(pred_t* p, pred::AttendArgs& a, const pred_kv_cache* cache, const pred_bf16* q, const int32_t* block_tables,
           int64_t n_blocks, const int32_t* kv_len, const int32_t* draft_len, float scale, pred_bf16* out, float* lse,
           void* workspace, size_t ws_bytes, void* stream, const char* what) {
    int rc;
    if ((rc = check_cache(p, cache, &a.cache, what)) || (rc = check_counts(p, n_blocks, a.S, what))) return rc;
    if (p->d.head_dim > kMostHead)
        return fail(PRED_ERR_UNSUPPORTED, "%s: head_dim (%d) above %d", what, p->d.head_dim, kMostHead);
    if (!block_tables && n_blocks > p->d.max_blocks)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: %lld blocks without a table, max_blocks %lld", what, (long long)n_blocks,
                    (long long)p->d.max_blocks);
    if (!std::isfinite(scale)) return fail(PRED_ERR_OUT_OF_RANGE, "%s: scale must be finite", what);
    if (a.S == 0) return ok();
    if (!q || !out) return fail(PRED_ERR_NULL_ARG, "%s: q or out is NULL", what);
    if (!pred::aligned16(q) || !pred::aligned16(out))
        return fail(PRED_ERR_UNSUPPORTED, "%s: q and out must be 16-byte aligned", what);
    // a row's queries are read by several workgroups, and its output may be written before the last of them starts
    const uint64_t bytes = (uint64_t)a.S * a.M * p->d.num_q_heads * p->d.head_dim * 2;
    const uint64_t from = (uint64_t)(uintptr_t)q, to = (uint64_t)(uintptr_t)out;
    if (from < to + bytes && to < from + bytes) return fail(PRED_ERR_OUT_OF_RANGE, "%s: out overlaps q", what);
    const size_t need = n_blocks > 0 ? pred::attend_workspace_bytes(a) : 0;
    if (need > 0 && (!workspace || ws_bytes < need))
        return fail(PRED_ERR_WORKSPACE, "%s needs a %zu-byte workspace (%zu given)", what, need,
                    workspace ? ws_bytes : (size_t)0);
    if (need > 0 && !pred::aligned16(workspace))
        return fail(PRED_ERR_WORKSPACE, "%s: the workspace must be 16-byte aligned", what);
    a.q = q;
    a.tables = block_tables;
    a.kv_len = kv_len;
    a.draft = draft_len;
    a.out = out;
    a.lse = lse;
    a.ws = workspace;
    a.scale = scale;
    const hipError_t e = pred::launch_attend(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, what);
    return ok();
}

int check_heads(int64_t n_tokens, int32_t n_heads, const char* what) {
    if (n_tokens < 0 || n_heads < 0 || n_heads > 65536)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: n_tokens (%lld) < 0 or n_heads (%d) outside [0, 65536]", what,
                    (long long)n_tokens, n_heads);
    return PRED_OK;
}

int check_in_place(const void* x, int64_t x_stride, const void* out, int64_t out_stride, const char* what,
                   const char* x_name, const char* out_name) {
    if (x == out && x_stride != out_stride)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: in place, %s and %s need one stride (%lld, %lld)", what, x_name,
                    out_name, (long long)x_stride, (long long)out_stride);
    return PRED_OK;
}

// New tokens into a cache: queries (unless `queries` is false) and keys normed
// where a norm is on, turned where rope is not NULL.
int store_rows(pred_t* p, const pred::HeadNorm& q_norm, const pred::HeadNorm& k_norm, const pred_rope* rope,
               const pred_bf16* q, int64_t q_stride, const pred_bf16* k, int64_t k_stride, const pred_bf16* v,
               int64_t v_stride, int64_t n_tokens, const int32_t* positions, const int64_t* slots,
               const pred_kv_cache* cache, pred_bf16* q_out, void* stream, bool queries, const char* what) {
    pred::CacheView view;
    int rc = check_cache(p, cache, &view, what);
    if (rc == 0) rc = check_store(cache, what);
    if (rc) return rc;
    if (n_tokens < 0) return fail(PRED_ERR_OUT_OF_RANGE, "%s: n_tokens (%lld) < 0", what, (long long)n_tokens);
    if (n_tokens == 0) return ok();
    if ((rope && !positions) || !slots) return fail(PRED_ERR_NULL_ARG, "%s: positions or slots is NULL", what);
    const pred_dims& d = p->d;
    const int64_t out_stride = (int64_t)d.num_q_heads * d.head_dim;
    if (queries && (rc = check_rows(p, q, q_stride, d.num_q_heads, what, "q"))) return rc;
    if ((rc = check_rows(p, k, k_stride, d.num_kv_heads, what, "k"))) return rc;
    if ((rc = check_rows(p, v, v_stride, d.num_kv_heads, what, "v"))) return rc;
    if (queries && (rc = check_rows(p, q_out, out_stride, d.num_q_heads, what, "q_out"))) return rc;
    if (queries && q == q_out && q_stride != out_stride)
        return fail(PRED_ERR_OUT_OF_RANGE, "%s: in place, q's stride (%lld) must be %lld", what, (long long)q_stride,
                    (long long)out_stride);
    if (d.num_q_heads > 65536 || d.num_kv_heads > 65536)
        return fail(PRED_ERR_UNSUPPORTED, "%s: more than 65536 heads", what);
    pred::NormArgs a{rope_args(p, rope, positions, n_tokens), q_norm, k_norm};
    a.rows.q = q;
    a.rows.k = k;
    a.rows.v = v;
    a.rows.out = q_out;
    a.rows.q_stride = q_stride;
    a.rows.k_stride = k_stride;
    a.rows.v_stride = v_stride;
    a.rows.out_stride = out_stride;
    a.rows.Hq = queries ? d.num_q_heads : 0;
    a.rows.Hk = d.num_kv_heads;
    a.rows.slots = slots;
    a.rows.cache = view;
    // rope.hip's kernels turn two pieces a lane and keep a cosine for both; they have no norms and no 4-bit rows
    const bool plain = rope && !q_norm.on && !k_norm.on && !view.fp4;
    const hipError_t e = plain ? pred::launch_rotate(a.rows, (hipStream_t)stream)
                               : pred::launch_norm_rotate(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, what);
    return ok();
}

}  // namespace

extern "C" {

int pred_rope_turns(int32_t rot_dim, double theta, const pred_rope_scaling* scaling, uint64_t* turns, float* mscale) {
    const pred_rope_scaling none = {PRED_ROPE_NONE, 1.0, 0.0, 0.0, 0.0};
    const pred_rope_scaling sc = scaling ? *scaling : none;
    if (!turns) return fail(PRED_ERR_NULL_ARG, "turns is NULL");
    if (rot_dim < 2 || (rot_dim & 1) || rot_dim > 65536)
        return fail(PRED_ERR_OUT_OF_RANGE, "rot_dim (%d) must be even and in [2, 65536]", rot_dim);
    if (!(theta > 1.0) || std::isinf(theta)) return fail(PRED_ERR_OUT_OF_RANGE, "theta must be above 1 and finite");
    if (sc.kind < PRED_ROPE_NONE || sc.kind > PRED_ROPE_YARN)
        return fail(PRED_ERR_OUT_OF_RANGE, "rope scaling kind %d is not one of PRED_ROPE_*", sc.kind);
    if (sc.kind != PRED_ROPE_NONE && (!(sc.factor > 0.0) || std::isinf(sc.factor)))
        return fail(PRED_ERR_OUT_OF_RANGE, "rope scaling factor must be positive and finite");
    if (sc.kind == PRED_ROPE_NTK && rot_dim == 2)
        return fail(PRED_ERR_OUT_OF_RANGE, "PRED_ROPE_NTK needs rot_dim above 2");
    const bool finite = std::isfinite(sc.low) && std::isfinite(sc.high) && std::isfinite(sc.original_length);
    if (sc.kind == PRED_ROPE_LLAMA3 && !(finite && sc.low > 0.0 && sc.high > sc.low && sc.original_length > 0.0))
        return fail(PRED_ERR_OUT_OF_RANGE, "PRED_ROPE_LLAMA3 needs 0 < low < high and original_length > 0");
    if (sc.kind == PRED_ROPE_YARN && !(finite && sc.low > 0.0 && sc.high > 0.0 && sc.original_length > 0.0))
        return fail(PRED_ERR_OUT_OF_RANGE, "PRED_ROPE_YARN needs low, high and original_length > 0");

    const double two_pi = 6.28318530717958647692;
    if (sc.kind == PRED_ROPE_NTK) theta *= std::pow(sc.factor, (double)rot_dim / (rot_dim - 2));
    double ramp_a = 0.0, ramp_b = 0.0;
    if (sc.kind == PRED_ROPE_YARN) {
        const double per = rot_dim / (2.0 * std::log(theta));
        ramp_a = std::fmax(std::floor(per * std::log(sc.original_length / (two_pi * sc.high))), 0.0);
        ramp_b = std::fmin(std::ceil(per * std::log(sc.original_length / (two_pi * sc.low))), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (sc.kind == PRED_ROPE_LINEAR) f /= sc.factor;
        if (sc.kind == PRED_ROPE_LLAMA3) {
            const double per_original = sc.original_length * f / two_pi;     // original_length / wavelength
            if (per_original < sc.low) f /= sc.factor;
            else if (per_original <= sc.high) {
                const double m = (per_original - sc.low) / (sc.high - sc.low);
                f = (1.0 - m) * f / sc.factor + m * f;
            }
        }
        if (sc.kind == PRED_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - ramp_a) / std::fmax(ramp_b - ramp_a, 0.001), 0.0), 1.0);
            f = f / sc.factor * ramp + f * (1.0 - ramp);
        }
        // whole turns add nothing; the fraction times 2^64 stays below 2^64 after rounding because a double
        // below 1 is at most 1 - 2^-53
        double turn = f / two_pi;
        turn -= std::floor(turn);
        turns[i] = turn < 1.0 ? (uint64_t)std::ldexp(turn, 64) : 0;
    }
    if (mscale) *mscale = sc.kind == PRED_ROPE_YARN ? (float)(0.1 * std::log(sc.factor) + 1.0) : 1.f;
    return ok();
}

int pred_rotate(pred_t* p, const pred_rope* rope, const pred_bf16* x, int64_t x_stride, int64_t n_tokens,
                int32_t n_heads, const int32_t* positions, pred_bf16* out, int64_t out_stride, void* stream) {
    int rc = check_handle(p, "rotate");
    if (rc == 0) rc = check_rope(p, rope, "rotate");
    if (rc) return rc;
    if ((rc = check_heads(n_tokens, n_heads, "rotate"))) return rc;
    if (n_tokens == 0 || n_heads == 0) return ok();
    if (!positions) return fail(PRED_ERR_NULL_ARG, "rotate: positions is NULL");
    if ((rc = check_rows(p, x, x_stride, n_heads, "rotate", "x"))) return rc;
    if ((rc = check_rows(p, out, out_stride, n_heads, "rotate", "out"))) return rc;
    if ((rc = check_in_place(x, x_stride, out, out_stride, "rotate", "x", "out"))) return rc;
    pred::RopeArgs a = rope_args(p, rope, positions, n_tokens);
    a.q = x;
    a.out = out;
    a.q_stride = x_stride;
    a.out_stride = out_stride;
    a.Hq = n_heads;
    const hipError_t e = pred::launch_rotate(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "rotate launch");
    return ok();
}

int pred_rotate_store(pred_t* p, const pred_rope* rope, const pred_bf16* q, int64_t q_stride, const pred_bf16* k,
                      int64_t k_stride, const pred_bf16* v, int64_t v_stride, int64_t n_tokens,
                      const int32_t* positions, const int64_t* slots, const pred_kv_cache* cache, pred_bf16* q_out,
                      void* stream) {
    int rc = check_handle(p, "rotate_store");
    if (rc == 0) rc = check_rope(p, rope, "rotate_store");
    if (rc) return rc;
    if (rope->backward) return fail(PRED_ERR_UNSUPPORTED, "rotate_store: rope->backward must be 0");
    return store_rows(p, pred::HeadNorm{}, pred::HeadNorm{}, rope, q, q_stride, k, k_stride, v, v_stride, n_tokens,
                      positions, slots, cache, q_out, stream, true, "rotate_store");
}

int pred_norm_rotate_store(pred_t* p, const pred_norm* q_norm, const pred_norm* k_norm, const pred_rope* rope,
                           const pred_bf16* q, int64_t q_stride, const pred_bf16* k, int64_t k_stride,
                           const pred_bf16* v, int64_t v_stride, int64_t n_tokens, const int32_t* positions,
                           const int64_t* slots, const pred_kv_cache* cache, pred_bf16* q_out, void* stream) {
    const char* const what = "norm_rotate_store";
    pred::HeadNorm qn, kn;
    int rc = check_handle(p, what);
    if (rc == 0) rc = check_norm(p, q_norm, &qn, what);
    if (rc == 0) rc = check_norm(p, k_norm, &kn, what);
    if (rc == 0) rc = check_forward_rope(p, rope, what);
    if (rc) return rc;
    return store_rows(p, qn, kn, rope, q, q_stride, k, k_stride, v, v_stride, n_tokens, positions, slots, cache, q_out,
                      stream, true, what);
}

int pred_store(pred_t* p, const pred_bf16* k, int64_t k_stride, const pred_bf16* v, int64_t v_stride, int64_t n_tokens,
               const int64_t* slots, const pred_kv_cache* cache, void* stream) {
    pred::HeadNorm none;
    int rc = check_handle(p, "store");
    if (rc == 0) rc = check_norm(p, nullptr, &none, "store");
    if (rc) return rc;
    return store_rows(p, none, none, nullptr, nullptr, 0, k, k_stride, v, v_stride, n_tokens, nullptr, slots, cache,
                      nullptr, stream, false, "store");
}

int pred_load(pred_t* p, const pred_kv_cache* cache, int64_t n_tokens, const int64_t* slots, pred_bf16* k_out,
              pred_bf16* v_out, void* stream) {
    int rc = check_handle(p, "load");
    if (rc) return rc;
    pred::CacheView view;
    if ((rc = check_cache(p, cache, &view, "load"))) return rc;
    if (n_tokens < 0) return fail(PRED_ERR_OUT_OF_RANGE, "load: n_tokens (%lld) < 0", (long long)n_tokens);
    if (n_tokens == 0) return ok();
    if (!slots) return fail(PRED_ERR_NULL_ARG, "load: slots is NULL");
    const pred_dims& d = p->d;
    const int64_t out_stride = (int64_t)d.num_kv_heads * d.head_dim;
    if ((rc = check_rows(p, k_out, out_stride, d.num_kv_heads, "load", "k_out"))) return rc;
    if ((rc = check_rows(p, v_out, out_stride, d.num_kv_heads, "load", "v_out"))) return rc;
    // a lane counts 8 values of a token at a time, up to five times as far as the token goes, in 32 bits
    if (out_stride > 1ll << 30)
        return fail(PRED_ERR_UNSUPPORTED, "load: %d heads of %d are more than 2^30 values", d.num_kv_heads, d.head_dim);
    // (more tokens than a launch takes are refused by it)
    const uint64_t bytes = 2ull * out_stride * (n_tokens < 1ll << 26 ? n_tokens : 1ll << 26);
    const uint64_t at_k = (uint64_t)(uintptr_t)k_out, at_v = (uint64_t)(uintptr_t)v_out;
    if (at_k < at_v + bytes && at_v < at_k + bytes) return fail(PRED_ERR_OUT_OF_RANGE, "load: k_out overlaps v_out");
    pred::LoadArgs a{};
    a.cache = view;
    a.slots = slots;
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = p->err_dev;
    a.n_tokens = n_tokens;
    a.N = d.max_blocks;
    a.Hk = d.num_kv_heads;
    a.D = d.head_dim;
    a.B = d.block_size;
    const hipError_t e = pred::launch_load(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "load launch");
    return ok();
}

int pred_norm_rotate(pred_t* p, const pred_norm* norm, const pred_rope* rope, const pred_bf16* x, int64_t x_stride,
                     int64_t n_tokens, int32_t n_heads, const int32_t* positions, pred_bf16* out, int64_t out_stride,
                     void* stream) {
    const char* const what = "norm_rotate";
    pred::NormArgs a{};
    int rc = check_handle(p, what);
    if (rc == 0 && !norm) rc = fail(PRED_ERR_NULL_ARG, "%s: norm is NULL", what);
    if (rc == 0) rc = check_norm(p, norm, &a.q, what);
    if (rc == 0) rc = check_forward_rope(p, rope, what);
    if (rc == 0) rc = check_heads(n_tokens, n_heads, what);
    if (rc) return rc;
    if (n_tokens == 0 || n_heads == 0) return ok();
    if (rope && !positions) return fail(PRED_ERR_NULL_ARG, "%s: positions is NULL", what);
    if ((rc = check_rows(p, x, x_stride, n_heads, what, "x")) ||
        (rc = check_rows(p, out, out_stride, n_heads, what, "out")) ||
        (rc = check_in_place(x, x_stride, out, out_stride, what, "x", "out")))
        return rc;
    a.rows = rope_args(p, rope, positions, n_tokens);
    a.rows.q = x;
    a.rows.out = out;
    a.rows.q_stride = x_stride;
    a.rows.out_stride = out_stride;
    a.rows.Hq = n_heads;
    const hipError_t e = pred::launch_norm_rotate(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "norm_rotate launch");
    return ok();
}

size_t pred_norm_rotate_workspace_bytes(pred_t* p, int64_t n_tokens, int32_t n_heads) {
    if (!p || n_tokens < 1 || n_heads < 1 || n_heads > 65536 || p->d.head_dim > 512) return 0;
    return (size_t)pred::norm_grad_parts(n_tokens, n_heads, p->d.head_dim) * p->d.head_dim * sizeof(float);
}

int pred_norm_rotate_backward(pred_t* p, const pred_norm* norm, const pred_rope* rope, const pred_bf16* x,
                              int64_t x_stride, int64_t n_tokens, int32_t n_heads, const int32_t* positions,
                              const pred_bf16* dy, int64_t dy_stride, pred_bf16* dx, int64_t dx_stride, float* dweight,
                              void* workspace, size_t ws_bytes, void* stream) {
    const char* const what = "norm_rotate_backward";
    pred::NormGradArgs a{};
    int rc = check_handle(p, what);
    if (rc == 0 && !norm) rc = fail(PRED_ERR_NULL_ARG, "%s: norm is NULL", what);
    if (rc == 0) rc = check_norm(p, norm, &a.norm, what);
    if (rc == 0) rc = check_forward_rope(p, rope, what);
    if (rc == 0) rc = check_heads(n_tokens, n_heads, what);
    if (rc) return rc;
    const bool none = n_tokens == 0 || n_heads == 0;
    if (none && !dweight) return ok();
    if (!none) {
        if (rope && !positions) return fail(PRED_ERR_NULL_ARG, "%s: positions is NULL", what);
        if ((rc = check_rows(p, x, x_stride, n_heads, what, "x")) ||
            (rc = check_rows(p, dy, dy_stride, n_heads, what, "dy")) ||
            (rc = check_rows(p, dx, dx_stride, n_heads, what, "dx")) ||
            (rc = check_in_place(x, x_stride, dx, dx_stride, what, "x", "dx")) ||
            (rc = check_in_place(dy, dy_stride, dx, dx_stride, what, "dy", "dx")))
            return rc;
        const size_t need = dweight ? pred_norm_rotate_workspace_bytes(p, n_tokens, n_heads) : 0;
        if (need > 0 && (!workspace || ws_bytes < need))
            return fail(PRED_ERR_WORKSPACE, "%s needs a %zu-byte workspace (%zu given)", what, need,
                        workspace ? ws_bytes : (size_t)0);
        if (need > 0 && !pred::aligned16(workspace))
            return fail(PRED_ERR_WORKSPACE, "%s: the workspace must be 16-byte aligned", what);
    }
    a.rows = rope_args(p, rope, positions, none ? 0 : n_tokens);
    a.rows.backward = 1;
    a.rows.q = x;
    a.rows.q_stride = x_stride;
    a.rows.out = dx;
    a.rows.out_stride = dx_stride;
    a.rows.Hq = n_heads;
    a.dy = dy;
    a.dy_stride = dy_stride;
    a.dweight = dweight;
    a.part = static_cast<float*>(workspace);
    const hipError_t e = pred::launch_norm_rotate_backward(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "norm_rotate_backward launch");
    return ok();
}

size_t pred_attend_workspace_bytes(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks) {
    if (!p || !attend_counts_ok(p, n_seqs, n_rows, n_blocks)) return 0;
    return pred::attend_workspace_bytes(attend_shape(p, n_seqs, n_rows, n_blocks));
}

const char* pred_attend_kernel_name(pred_t* p, const pred_kv_cache* cache, int32_t n_rows, int32_t with_block_lse) {
    if (!p) {
        fail(PRED_ERR_NULL_ARG, "attend_kernel_name: predictor is NULL");
        return nullptr;
    }
    pred::CacheView view;
    if (check_cache(p, cache, &view, "attend_kernel_name") || check_n_rows(n_rows, "attend_kernel_name"))
        return nullptr;
    if (p->d.head_dim > kMostHead) {
        fail(PRED_ERR_UNSUPPORTED, "attend_kernel_name: head_dim (%d) above %d", p->d.head_dim, kMostHead);
        return nullptr;
    }
    pred::AttendArgs a = attend_shape(p, 1, n_rows, 1);
    a.cache = view;
    float any;
    a.block_lse = with_block_lse ? &any : nullptr;
    ok();
    return pred::attend_kernel_name(a);
}

int pred_attend(pred_t* p, const pred_kv_cache* cache, const pred_bf16* q, int32_t n_rows, const uint64_t* tree,
                const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs, const int32_t* kv_len,
                const int32_t* draft_len, float scale, pred_bf16* out, float* lse, float* block_lse, void* workspace,
                size_t ws_bytes, void* stream) {
    int rc = check_handle(p, "attend");
    if (rc == 0) rc = check_n_rows(n_rows, "attend");
    if (rc) return rc;
    pred::AttendArgs a = attend_shape(p, n_seqs, n_rows, n_blocks);
    a.tree = tree;
    a.block_lse = block_lse;
    return attend(p, a, cache, q, block_tables, n_blocks, kv_len, draft_len, scale, out, lse, workspace, ws_bytes, stream,
                  "attend");
}

size_t pred_attend_window_workspace_bytes(pred_t* p, int32_t n_seqs, int32_t n_rows, int64_t n_blocks, int32_t window,
                                          int32_t n_sinks) {
    if (!p || n_seqs < 1 || !window_rows_ok(p, n_rows) || n_blocks < 1 || n_blocks > kMostTokens / p->d.block_size ||
        window < 1 || n_sinks < 0)
        return 0;
    pred::AttendArgs a = attend_shape(p, n_seqs, n_rows, n_blocks);
    set_window(&a, window, n_sinks);
    return pred::attend_workspace_bytes(a);
}

const char* pred_attend_window_kernel_name(pred_t* p, const pred_kv_cache* cache, int32_t n_rows) {
    const char* const what = "attend_window_kernel_name";
    if (!p) {
        fail(PRED_ERR_NULL_ARG, "%s: predictor is NULL", what);
        return nullptr;
    }
    pred::CacheView view;
    if (check_cache(p, cache, &view, what) || check_window(p, n_rows, 1, 0, what)) return nullptr;
    if (p->d.head_dim > kMostHead) {
        fail(PRED_ERR_UNSUPPORTED, "%s: head_dim (%d) above %d", what, p->d.head_dim, kMostHead);
        return nullptr;
    }
    pred::AttendArgs a = attend_shape(p, 1, n_rows, 1);
    a.cache = view;
    set_window(&a, 1, 0);
    ok();
    return pred::attend_kernel_name(a);
}

int pred_attend_window(pred_t* p, const pred_kv_cache* cache, const pred_bf16* q, int32_t n_rows,
                       const int32_t* block_tables, int64_t n_blocks, int32_t n_seqs, const int32_t* kv_len,
                       const int32_t* row_len, int32_t window, int32_t n_sinks, float scale, pred_bf16* out, float* lse,
                       void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_handle(p, "attend_window");
    if (rc == 0) rc = check_window(p, n_rows, window, n_sinks, "attend_window");
    if (rc) return rc;
    pred::AttendArgs a = attend_shape(p, n_seqs, n_rows, n_blocks);
    set_window(&a, window, n_sinks);
    return attend(p, a, cache, q, block_tables, n_blocks, kv_len, row_len, scale, out, lse, workspace, ws_bytes, stream,
                  "attend_window");
}

int pred_accumulate_weight(pred_t* p, const float* lse, const float* block_lse, int32_t n_rows,
                           const uint64_t* accepted, const int32_t* kv_len, int64_t n_blocks, int32_t n_seqs,
                           float decay, const float* mass, float* mass_out, void* stream) {
    int rc = check_handle(p, "accumulate_weight");
    if (rc == 0) rc = check_counts(p, n_blocks, n_seqs, "accumulate_weight");
    if (rc == 0) rc = check_n_rows(n_rows, "accumulate_weight");
    if (rc) return rc;
    if (!std::isfinite(decay)) return fail(PRED_ERR_OUT_OF_RANGE, "accumulate_weight: decay must be finite");
    if (n_blocks == 0 || n_seqs == 0) return ok();
    if (!lse || !block_lse || !mass || !mass_out)
        return fail(PRED_ERR_NULL_ARG, "accumulate_weight: lse, block_lse, mass or mass_out is NULL");
    pred::WeightArgs a{};
    a.lse = lse;
    a.block_lse = block_lse;
    a.accepted = accepted;
    a.kv_len = kv_len;
    a.mass = mass;
    a.mass_out = mass_out;
    a.err = p->err_dev;
    a.decay = decay;
    a.n = n_blocks;
    a.S = n_seqs;
    a.M = n_rows;
    a.Hq = p->d.num_q_heads;
    a.B = p->d.block_size;
    const hipError_t e = pred::launch_weight(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "accumulate_weight launch");
    return ok();
}

size_t pred_evict_workspace_bytes(int64_t n_blocks, int32_t n_seqs) {
    return pred::evict_workspace_bytes(n_blocks, n_seqs);
}

int pred_evict_blocks(pred_t* p, const int32_t* block_tables, const float* mass, const int32_t* kv_len,
                      int64_t n_blocks, int32_t n_seqs, int64_t budget, int32_t protect_first, int32_t protect_last,
                      int32_t* tables_out, float* mass_out, int32_t* kv_len_out, int32_t* evicted, void* workspace,
                      size_t ws_bytes, void* stream) {
    int rc = check_handle(p, "evict_blocks");
    if (rc == 0) rc = check_counts(p, n_blocks, n_seqs, "evict_blocks");
    if (rc) return rc;
    if (budget < 0 || protect_first < 0 || protect_last < 1)
        return fail(PRED_ERR_OUT_OF_RANGE,
                    "evict_blocks: budget (%lld) and protect_first (%d) must be >= 0 and protect_last (%d) >= 1",
                    (long long)budget, protect_first, protect_last);
    if (n_seqs == 0) return ok();
    if (!kv_len || !kv_len_out || !evicted)
        return fail(PRED_ERR_NULL_ARG, "evict_blocks: kv_len, kv_len_out or evicted is NULL");
    if (n_blocks > 0 && (!block_tables || !mass || !tables_out || !mass_out))
        return fail(PRED_ERR_NULL_ARG, "evict_blocks: a table or a mass is NULL");
    const size_t need = pred::evict_workspace_bytes(n_blocks, n_seqs);
    if (need > 0 && (!workspace || ws_bytes < need))
        return fail(PRED_ERR_WORKSPACE, "evict_blocks needs a %zu-byte workspace (%zu given)", need,
                    workspace ? ws_bytes : (size_t)0);
    if (need > 0 && !pred::aligned_to(workspace, 8))
        return fail(PRED_ERR_WORKSPACE, "evict_blocks: the workspace must be 8-byte aligned");
    pred::EvictArgs a{};
    a.tables = block_tables;
    a.mass = mass;
    a.kv_len = kv_len;
    a.tables_out = tables_out;
    a.mass_out = mass_out;
    a.kv_len_out = kv_len_out;
    a.evicted = evicted;
    a.ws = workspace;
    a.err = p->err_dev;
    a.n = n_blocks;
    a.budget = budget;
    a.S = n_seqs;
    a.B = p->d.block_size;
    a.first = protect_first;
    a.last = protect_last;
    const hipError_t e = pred::launch_evict(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "evict_blocks launch");
    return ok();
}

}  // extern "C"
