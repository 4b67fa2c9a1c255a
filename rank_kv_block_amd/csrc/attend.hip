// Attention of a sequence's newest tokens (one, or a tree of drafted ones) over
// its paged cache.
#include "common.h"
#include "kernels.h"

namespace pred {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// Start of a running maximum: finite, so that exp2(-inf - max) is 0 and not NaN
// for a masked score before the first real one.
constexpr float kLowest = -3.402823466e38f;

__device__ inline float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float log2_of(float x) { return __builtin_amdgcn_logf(x); }

// Which drafted tokens row i sees, a bit each.
__device__ inline uint64_t tree_word(const AttendArgs& a, int s, int i) {
    return a.tree ? a.tree[(int64_t)s * a.M + i] : ~0ull >> (63 - i);
}

// The lengths given for sequence s, checked once per sequence.
__device__ inline void check_lengths(const AttendArgs& a, int s, int len, int drafted) {
    if ((a.kv_len && a.kv_len[s] != len) || (a.draft && a.draft[s] != drafted)) atomicOr(a.err, DEVERR_LEN);
}

__device__ inline uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

__device__ inline float fp8_value(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }

// ---------------------------------------------------------------- plain kernel
//
// Any head size up to 256, any block size and strides: a workgroup per (row,
// query head), its four waves taking every fourth block.  A wave scores up to
// 64 tokens of a block at a time, a lane each, then adds their values with a
// lane per value.  Every query head reads its kv head's cache for itself, so
// this kernel is for the shapes the others do not take.
template <bool FP8>
__device__ inline float cache_value(const void* p, int64_t at) {
    if constexpr (FP8) return fp8_value(static_cast<const uint8_t*>(p)[at]);
    else return bf16_lo(static_cast<const uint16_t*>(p)[at]);
}

constexpr int kPlainHead = 256;     // largest head size

template <bool FP8>
__global__ __launch_bounds__(256) void attend_plain_kernel(AttendArgs a) {
    __shared__ float q_row[kPlainHead];
    __shared__ float part[4][kPlainHead];
    __shared__ float part_m[4], part_l[4];
    const int h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.M, s = blockIdx.x / a.Hq / a.M;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = kv_len_of(a.kv_len, s, (int64_t)a.n * a.B), drafted = draft_len_of(a, s, len);
    if (h == 0 && i == 0 && threadIdx.x == 0) check_lengths(a, s, len, drafted);
    const int ctx = len - drafted;
    const bool live = i < drafted;
    const uint64_t seen = tree_word(a, s, i);
    const int64_t q_at = (((int64_t)s * a.M + i) * a.Hq + h) * a.D;
    const float scale = a.scale * a.cache.k_scale * kLog2e;
    for (int d = threadIdx.x; d < a.D; d += 256) q_row[d] = bf16_lo(a.q[q_at + d]);
    __syncthreads();

    const int64_t head_off = (int64_t)(h / (a.Hq / a.Hk)) * a.cache.head_stride;
    const int used = (int)(((int64_t)len + a.B - 1) / a.B);
    float m = kLowest, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b = wave; b < used; b += 4) {
        const int64_t slot = a.tables ? a.tables[(int64_t)s * a.n + b] : b;
        const bool good = slot >= 0 && slot < a.N;
        if (!good && lane == 0) atomicOr(a.err, DEVERR_TABLE);
        float bm = kLowest, bl = 0.f;
        for (int t0 = 0; good && live && t0 < a.B && b * a.B + t0 < len; t0 += 64) {
            const int t = b * a.B + t0 + lane;
            const bool sees = t0 + lane < a.B && t < len && (t < ctx || ((seen >> (t - ctx)) & 1));
            const int64_t base = slot * a.cache.block_stride + t0 * a.cache.token_stride + head_off;
            float x = 0.f;
            if (sees) {
                const int64_t at = base + lane * a.cache.token_stride;
                for (int d = 0; d < a.D; ++d) x += q_row[d] * cache_value<FP8>(a.cache.k, at + d);
            }
            x = sees ? x * scale : -INFINITY;
            float top = x;
            for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            const float m_new = fmaxf(m, top), bm_new = fmaxf(bm, top);
            const float alpha = exp2_of(m - m_new);
            const float p = exp2_of(x - m_new);
            float sum = p, bsum = exp2_of(x - bm_new);
            for (int o = 32; o >= 1; o >>= 1) {
                sum += __shfl_xor(sum, o);
                bsum += __shfl_xor(bsum, o);
            }
            l = l * alpha + sum;
            bl = bl * exp2_of(bm - bm_new) + bsum;
            m = m_new;
            bm = bm_new;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] *= alpha;
            for (uint64_t todo = __ballot(sees); todo; todo &= todo - 1) {
                const int tok = __builtin_ctzll(todo);
                const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), tok));
                const int64_t at = base + tok * a.cache.token_stride;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (lane + 64 * e < a.D) acc[e] += w * cache_value<FP8>(a.cache.v, at + lane + 64 * e);
            }
        }
        if (a.block_lse && lane == 0)
            a.block_lse[(((int64_t)s * a.n + b) * a.M + i) * a.Hq + h] =
                bl > 0.f || bl != bl ? (bm + log2_of(bl)) * kLn2 : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][lane + 64 * e] = acc[e];
    if (lane == 0) {
        part_m[wave] = m;
        part_l[wave] = l;
    }
    __syncthreads();
    const float top = fmaxf(fmaxf(part_m[0], part_m[1]), fmaxf(part_m[2], part_m[3]));
    float total = 0.f, value = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = exp2_of(part_m[w] - top);
        total += f * part_l[w];
        value += f * part[w][threadIdx.x];
    }
    const bool none = total == 0.f;
    if ((int)threadIdx.x < a.D) a.out[q_at + threadIdx.x] = to_bf16(none ? 0.f : value * a.cache.v_scale / total);
    if (a.lse && threadIdx.x == 0)
        a.lse[((int64_t)s * a.M + i) * a.Hq + h] = none ? -INFINITY : (top + log2_of(total)) * kLn2;
}

}  // namespace

size_t attend_workspace_bytes(const AttendArgs&) { return 0; }

const char* attend_kernel_name(const AttendArgs&) { return "attend_plain_kernel"; }

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    const int64_t groups = (int64_t)a.S * a.M;
    if (groups > 0x7FFFFFFF / a.Hq) return hipErrorInvalidConfiguration;
    const uint32_t grid = (uint32_t)(groups * a.Hq);
    if (a.cache.fp8) attend_plain_kernel<true><<<grid, 256, 0, stream>>>(a);
    else attend_plain_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace pred
