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
    if (c->dtype != PRED_KV_BF16 && c->dtype != PRED_KV_FP8)
        return fail(PRED_ERR_UNSUPPORTED, "%s: cache dtype %d is not PRED_KV_BF16 or PRED_KV_FP8", what, c->dtype);
    const pred_dims& d = p->d;
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
    if (c->dtype == PRED_KV_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f))
        return fail(PRED_ERR_UNSUPPORTED, "%s: a bf16 cache has scales of 1", what);
    *out = pred::CacheView{c->k, c->v, bs, ts, hs, c->dtype == PRED_KV_FP8, c->k_scale, c->v_scale};
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

pred::RopeArgs rope_args(pred_t* p, const pred_rope* r, const int32_t* positions, int64_t n_tokens) {
    pred::RopeArgs a{};
    a.turns = r->turns;
    a.rot = r->rot_dim;
    a.interleaved = r->interleaved != 0;
    a.backward = r->backward != 0;
    a.mscale = r->mscale;
    a.positions = positions;
    a.n_tokens = n_tokens;
    a.D = p->d.head_dim;
    a.N = p->d.max_blocks;
    a.B = p->d.block_size;
    a.err = p->err_dev;
    return a;
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
    if (n_tokens < 0 || n_heads < 0 || n_heads > 65536)
        return fail(PRED_ERR_OUT_OF_RANGE, "rotate: n_tokens (%lld) < 0 or n_heads (%d) outside [0, 65536]",
                    (long long)n_tokens, n_heads);
    if (n_tokens == 0 || n_heads == 0) return ok();
    if (!positions) return fail(PRED_ERR_NULL_ARG, "rotate: positions is NULL");
    if ((rc = check_rows(p, x, x_stride, n_heads, "rotate", "x"))) return rc;
    if ((rc = check_rows(p, out, out_stride, n_heads, "rotate", "out"))) return rc;
    if (x == out && x_stride != out_stride)
        return fail(PRED_ERR_OUT_OF_RANGE, "rotate: in place, x and out need one stride (%lld, %lld)",
                    (long long)x_stride, (long long)out_stride);
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
    pred::CacheView view;
    if ((rc = check_cache(p, cache, &view, "rotate_store"))) return rc;
    if (cache->k == cache->v) return fail(PRED_ERR_OUT_OF_RANGE, "rotate_store: the cache's k and v are one");
    if (n_tokens < 0) return fail(PRED_ERR_OUT_OF_RANGE, "rotate_store: n_tokens (%lld) < 0", (long long)n_tokens);
    if (n_tokens == 0) return ok();
    if (!positions || !slots) return fail(PRED_ERR_NULL_ARG, "rotate_store: positions or slots is NULL");
    const pred_dims& d = p->d;
    const int64_t out_stride = (int64_t)d.num_q_heads * d.head_dim;
    if ((rc = check_rows(p, q, q_stride, d.num_q_heads, "rotate_store", "q"))) return rc;
    if ((rc = check_rows(p, k, k_stride, d.num_kv_heads, "rotate_store", "k"))) return rc;
    if ((rc = check_rows(p, v, v_stride, d.num_kv_heads, "rotate_store", "v"))) return rc;
    if ((rc = check_rows(p, q_out, out_stride, d.num_q_heads, "rotate_store", "q_out"))) return rc;
    if (q == q_out && q_stride != out_stride)
        return fail(PRED_ERR_OUT_OF_RANGE, "rotate_store: in place, q's stride (%lld) must be %lld",
                    (long long)q_stride, (long long)out_stride);
    if (d.num_q_heads > 65536 || d.num_kv_heads > 65536)
        return fail(PRED_ERR_UNSUPPORTED, "rotate_store: more than 65536 heads");
    pred::RopeArgs a = rope_args(p, rope, positions, n_tokens);
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = out_stride;
    a.Hq = d.num_q_heads;
    a.Hk = d.num_kv_heads;
    a.slots = slots;
    a.cache = view;
    const hipError_t e = pred::launch_rotate(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "rotate_store launch");
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
    if (rc) return rc;
    pred::CacheView view;
    if ((rc = check_cache(p, cache, &view, "attend")) || (rc = check_counts(p, n_blocks, n_seqs, "attend")) ||
        (rc = check_n_rows(n_rows, "attend")))
        return rc;
    if (p->d.head_dim > kMostHead)
        return fail(PRED_ERR_UNSUPPORTED, "attend: head_dim (%d) above %d", p->d.head_dim, kMostHead);
    if (!block_tables && n_blocks > p->d.max_blocks)
        return fail(PRED_ERR_OUT_OF_RANGE, "attend: %lld blocks without a table, max_blocks %lld", (long long)n_blocks,
                    (long long)p->d.max_blocks);
    if (!std::isfinite(scale)) return fail(PRED_ERR_OUT_OF_RANGE, "attend: scale must be finite");
    if (n_seqs == 0) return ok();
    if (!q || !out) return fail(PRED_ERR_NULL_ARG, "attend: q or out is NULL");
    if (!pred::aligned16(q) || !pred::aligned16(out))
        return fail(PRED_ERR_UNSUPPORTED, "attend: q and out must be 16-byte aligned");
    // a row's queries are read by several workgroups, and its output may be written before the last of them starts
    const uint64_t bytes = (uint64_t)n_seqs * n_rows * p->d.num_q_heads * p->d.head_dim * 2;
    const uint64_t from = (uint64_t)(uintptr_t)q, to = (uint64_t)(uintptr_t)out;
    if (from < to + bytes && to < from + bytes) return fail(PRED_ERR_OUT_OF_RANGE, "attend: out overlaps q");
    pred::AttendArgs a = attend_shape(p, n_seqs, n_rows, n_blocks);
    const size_t need = n_blocks > 0 ? pred::attend_workspace_bytes(a) : 0;
    if (need > 0 && (!workspace || ws_bytes < need))
        return fail(PRED_ERR_WORKSPACE, "attend needs a %zu-byte workspace (%zu given)", need,
                    workspace ? ws_bytes : (size_t)0);
    if (need > 0 && !pred::aligned16(workspace))
        return fail(PRED_ERR_WORKSPACE, "attend: the workspace must be 16-byte aligned");
    a.cache = view;
    a.q = q;
    a.tree = tree;
    a.tables = block_tables;
    a.kv_len = kv_len;
    a.draft = draft_len;
    a.out = out;
    a.lse = lse;
    a.block_lse = block_lse;
    a.ws = workspace;
    a.scale = scale;
    const hipError_t e = pred::launch_attend(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "attend launch");
    return ok();
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
