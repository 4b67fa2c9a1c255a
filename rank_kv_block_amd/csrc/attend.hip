// Attention of a sequence's newest tokens (one, or a tree of drafted ones) over
// its paged cache.
#include <type_traits>

#include "attend.h"
#include "common.h"
#include "kernels.h"

namespace pred {
namespace attend {
namespace {

// ---------------------------------------------------------------- plain kernel
//
// Any head size up to 256, any block size and strides: a workgroup per (row,
// query head), its four waves taking every fourth block.  A wave scores up to
// 64 tokens of a block at a time, a lane each, then adds their values with a
// lane per value.  Every query head reads its kv head's cache for itself, so
// this kernel is for the shapes the others do not take (16 sequences of 8192
// tokens, 32 queries of 64 over 8 e4m3 heads: 2021 us, the tree kernel 39; one
// sequence of 16384 tokens, 32 queries over 8 bf16 heads: 4.9 ms at a head size
// of 80 and 13.1 ms at 256, the stream kernel 18 us at 128).
template <Held HELD>
__device__ inline float cache_value(const void* p, const uint8_t* scales, int64_t at) {
    if constexpr (HELD == FP4) {
        const uint32_t byte = static_cast<const uint8_t*>(p)[at / 2];
        const auto pair = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(byte, __uint_as_float((uint32_t)scales[at / 32] << 23), 0);
        return at % 2 ? pair[1] : pair[0];
    } else if constexpr (HELD == FP8) {
        return fp8_value(static_cast<const uint8_t*>(p)[at]);
    } else {
        return bf16_lo(static_cast<const uint16_t*>(p)[at]);
    }
}

constexpr int kPlainHead = 256;     // largest head size

template <Held HELD, bool WINDOW>
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
    const uint64_t seen = WINDOW ? 0 : tree_word(a, s, i);
    const int pos = ctx + i, first = pos - a.window + 1;       // with a window
    auto sees_token = [&](int t) {
        if constexpr (WINDOW) return t <= pos && (t >= first || t < a.sinks);
        else return t < ctx || ((seen >> (t - ctx)) & 1);
    };
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
        if (WINDOW && (b * a.B > pos || (b * a.B >= a.sinks && (b + 1) * a.B <= first))) continue;     // no token of it seen
        // (with a window the entries that count are those of tokens some row sees, and each live row meets its own)
        if (!good && lane == 0 && (!WINDOW || live)) atomicOr(a.err, DEVERR_TABLE);
        float bm = kLowest, bl = 0.f;
        for (int t0 = 0; good && live && t0 < a.B && b * a.B + t0 < len; t0 += 64) {
            const int t = b * a.B + t0 + lane;
            const bool sees = t0 + lane < a.B && t < len && sees_token(t);
            const int64_t base = slot * a.cache.block_stride + t0 * a.cache.token_stride + head_off;
            float x = 0.f;
            if (sees) {
                const int64_t at = base + lane * a.cache.token_stride;
                for (int d = 0; d < a.D; ++d) x += q_row[d] * cache_value<HELD>(a.cache.k, a.cache.k_scales, at + d);
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
                    if (lane + 64 * e < a.D) acc[e] += w * cache_value<HELD>(a.cache.v, a.cache.v_scales, at + lane + 64 * e);
            }
        }
        if (a.block_lse && lane == 0)
            a.block_lse[(((int64_t)s * a.n + b) * a.M + i) * a.Hq + h] =
                bl <= 0.f ? -INFINITY : (bm + log2_of(bl)) * kLn2;
    }
    if constexpr (HELD == BF16) {
        const float lost = acc[0] * 0.f + acc[1] * 0.f + acc[2] * 0.f + acc[3] * 0.f;      // NaN where a sum is not finite
        if (__ballot(lost != 0.f) && l == l) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            for (int b = wave; b < used; b += 4) {
                const int64_t slot = a.tables ? a.tables[(int64_t)s * a.n + b] : b;
                if (slot < 0 || slot >= a.N) continue;
                for (int t0 = 0; t0 < a.B && b * a.B + t0 < len; ++t0) {
                    const int t = b * a.B + t0;
                    if (!sees_token(t)) continue;
                    const int64_t at = slot * a.cache.block_stride + t0 * a.cache.token_stride + head_off;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (lane + 64 * e < a.D) sum[e] += not_finite(cache_value<HELD>(a.cache.v, a.cache.v_scales, at + lane + 64 * e));
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = sum[e] == 0.f ? acc[e] : sum[e];
        }
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
    if (value != value)
        value = part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
    const bool none = total == 0.f;
    if ((int)threadIdx.x < a.D) a.out[q_at + threadIdx.x] = to_bf16(none ? 0.f : value * a.cache.v_scale / total);
    if (a.lse && threadIdx.x == 0)
        a.lse[((int64_t)s * a.M + i) * a.Hq + h] = none ? -INFINITY : (top + log2_of(total)) * kLn2;
}

// Joins a row's runs: out = sum_r 2^(m_r - m) o_r / sum_r 2^(m_r - m) l_r, for a
// row (sequence, drafted row, query head) that has more than one.  Bound: the
// partial sums, and a launch's latency for few rows.
struct JoinRow {
    int h, s, runs, in_group;       // runs: 0 for a row past the draft, which has no partial sums
    bool wanted;                    // else its items wrote the result
    int64_t slot, step;             // of its first run, and from one to the next
};
__device__ inline JoinRow join_row(const AttendArgs& a, const Plan& pl, uint32_t row) {
    JoinRow j;
    j.h = (int)(row % (uint32_t)a.Hq);
    const int i = (int)(row / (uint32_t)a.Hq % (uint32_t)a.M);
    j.s = (int)(row / (uint32_t)a.Hq / (uint32_t)a.M);
    const Share share = shares_of(a)[j.s];
    const int g = a.Hq / a.Hk, r = i * g + j.h % g, drafted = draft_len_of(a, j.s, share.len);
    int runs = share.runs;
    if (pl.chunk) runs = chunk_runs(chunk_span(a, pl, share.len, drafted, r / pl.rows), share.run);
    j.wanted = runs > 1;
    j.runs = j.wanted && i < drafted ? runs : 0;
    j.in_group = r % pl.rows;
    j.step = (int64_t)a.Hk * share.groups;
    j.slot = (int64_t)share.first * a.Hk + (int64_t)(j.h / g) * share.groups + r / pl.rows;
    return j;
}
// 4 values of a row's sums where one of them is NaN: the runs' without their factors
__device__ inline float4 join_not_finite(const AttendArgs& a, const Plan& pl, const JoinRow& j, int D, int d4, float4 v) {
    if (!(v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w)) return v;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < j.runs; ++x) {
        const float4 o = reinterpret_cast<const float4*>(part_sums(a, pl, j.slot + x * j.step) + j.in_group * D)[d4];
        sum = make_float4(sum.x + o.x, sum.y + o.y, sum.z + o.z, sum.w + o.w);
    }
    return make_float4(v.x != v.x ? sum.x : v.x, v.y != v.y ? sum.y : v.y, v.z != v.z ? sum.z : v.z, v.w != v.w ? sum.w : v.w);
}
// 4 values of a row from its sums (v, l, m), the lse by the first lane
__device__ inline void join_store(const AttendArgs& a, int D, uint32_t row, int d4, float4 v, float l, float m) {
    const bool none = l == 0.f;
    const float f = none ? 0.f : a.cache.v_scale / l;
    const uint2 w = make_uint2(bf16_pair(v.x * f, v.y * f), bf16_pair(v.z * f, v.w * f));
    *reinterpret_cast<uint2*>(a.out + (int64_t)row * D + 4 * d4) = none ? make_uint2(0, 0) : w;
    if (a.lse && d4 == 0) a.lse[row] = none ? -INFINITY : (m + log2_of(l)) * kLn2;
}

// Rows of few runs: D / 4 lanes a row, 4 values each, that read the row's
// (maximum, total) for themselves, kAhead runs in flight.  65536 rows, half of
// them live, of 2 to 4 runs: 21 us (38 with a wave a row; 8 runs in flight 24).
template <int D>
__global__ __launch_bounds__(256) void attend_join_rows_kernel(AttendArgs a, Plan pl, uint32_t rows) {
    constexpr int lanes = D / 4, kAhead = 4;
    const int d4 = threadIdx.x % lanes;
    if (pl.whole_from > 0 && shares_of(a)[0].runs == 1) return;      // (one sequence's walks)
    for (uint32_t row = blockIdx.x * (256 / lanes) + threadIdx.x / lanes; row < rows; row += gridDim.x * (256 / lanes)) {
        const JoinRow j = join_row(a, pl, row);
        if (!j.wanted) continue;
        float m = kLowest, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = 0; x0 < j.runs; x0 += kAhead) {
            float4 o[kAhead];
            float2 st[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                st[e] = make_float2(kLowest, 0.f);
                o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x0 + e >= j.runs) continue;
                const int64_t slot = j.slot + (x0 + e) * j.step;
                st[e] = part_stats(a, pl, slot)[j.in_group];
                o[e] = reinterpret_cast<const float4*>(part_sums(a, pl, slot) + j.in_group * D)[d4];
            }
            float top = m;
#pragma unroll
            for (int e = 0; e < kAhead; ++e) top = fmaxf(top, st[e].x);
            const float alpha = exp2_of(m - top);
            m = top;
            l *= alpha;
            v = make_float4(v.x * alpha, v.y * alpha, v.z * alpha, v.w * alpha);
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const float f = exp2_of(st[e].x - top);
                l += f * st[e].y;
                v = make_float4(v.x + f * o[e].x, v.y + f * o[e].y, v.z + f * o[e].z, v.w + f * o[e].w);
            }
        }
        join_store(a, D, row, d4, join_not_finite(a, pl, j, D, d4, v), l, m);
    }
}

// Rows of many runs: a workgroup each, wave w taking runs w, w + 4, ..: a lane
// reads one run's (maximum, total), then the wave adds the runs' sums, 4 values
// a lane and 64 / (D / 4) runs at a time.  32 rows of 64 runs: 4.7 us.
template <int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, Plan pl) {
    __shared__ float4 sums[4][64];
    __shared__ float2 stats[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t row = blockIdx.x;        // [S, M, Hq]
    const JoinRow j = join_row(a, pl, row);
    if (!j.wanted) return;
    constexpr int lanes = D / 4, groups = 64 / lanes, kAhead = 8;       // kAhead loads in flight a lane
    const int part = lane / lanes, d4 = lane % lanes;
    float m = kLowest, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    // 64 at a time for the statistics, groups * kAhead for the sums
    const int mine = (j.runs - wave + 3) / 4;
    for (int x0 = 0; x0 < mine; x0 += 64) {
        auto slot_at = [&](int x) { return j.slot + (int64_t)(wave + 4 * x) * j.step; };
        const int count = mine - x0 < 64 ? mine - x0 : 64;
        const float2 st = lane < count ? part_stats(a, pl, slot_at(x0 + lane))[j.in_group] : make_float2(kLowest, 0.f);
        float top = m, weight = 0.f;
        for (int y0 = 0; y0 < count; y0 += groups * kAhead) {
            float4 o[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int x = y0 + e * groups + part;
                o[e] = reinterpret_cast<const float4*>(part_sums(a, pl, slot_at(x0 + (x < count ? x : 0))) +
                                                       j.in_group * D)[d4];
            }
            if (y0 == 0) {
                top = fmaxf(m, st.x);
                for (int e = 32; e >= 1; e >>= 1) top = fmaxf(top, __shfl_xor(top, e));
                const float alpha = exp2_of(m - top);
                weight = lane < count ? exp2_of(st.x - top) : 0.f;
                m = top;
                l = l * alpha + weight * st.y;
                v = make_float4(v.x * alpha, v.y * alpha, v.z * alpha, v.w * alpha);
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int x = y0 + e * groups + part;
                const float f = __shfl(weight, x & 63);
                if (x < count) v = make_float4(v.x + f * o[e].x, v.y + f * o[e].y, v.z + f * o[e].z, v.w + f * o[e].w);
            }
        }
    }
    for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o);
    for (int o = lanes; o < 64; o <<= 1) {
        v.x += __shfl_xor(v.x, o);
        v.y += __shfl_xor(v.y, o);
        v.z += __shfl_xor(v.z, o);
        v.w += __shfl_xor(v.w, o);
    }
    sums[wave][lane] = v;
    if (lane == 0) stats[wave] = make_float2(m, l);
    __syncthreads();
    if (wave != 0) return;
    const float own = m;
    for (int w = 1; w < 4; ++w) m = fmaxf(m, stats[w].x);
    const float f = exp2_of(own - m);
    l *= f;
    v.x *= f;
    v.y *= f;
    v.z *= f;
    v.w *= f;
    for (int w = 1; w < 4; ++w) {
        const float fw = exp2_of(stats[w].x - m);
        const float4 o = sums[w][lane];
        l += fw * stats[w].y;
        v.x += fw * o.x;
        v.y += fw * o.y;
        v.z += fw * o.z;
        v.w += fw * o.w;
    }
    if (part == 0) join_store(a, D, row, d4, join_not_finite(a, pl, j, D, d4, v), l, m);
}

// ---------------------------------------------------------------- stream kernel
//
// Up to 32 queries per kv head (a token, or a small draft): HBM bound, every
// key and value read once for each 16 queries.  Each of a workgroup's four waves
// works alone on every fourth tile of 32 tokens, from loads to sums, with no LDS
// and no barrier, and the waves' sums meet at the end.
//
// A wave-load takes 1 KiB, whole rows of TPL tokens (row = a token's head, RB
// bytes).  Both products run on v_mfma_f32_16x16x32_bf16, queries as the second
// operand (column n = lane % 16 of both results is query n, c = lane / 16):
//   scores  row m of the first operand is (token m / H, part m % H) of a load,
//           H = RB / 64: lane (m, c) holds 16 bytes, piece 4 (m % H) + c of
//           token m / H, so the wave-load is contiguous.  MFMA j multiplies
//           by part j of the queries; of its 16 results rows with m % H = j
//           count, and lane (n, c) keeps tokens W c .. W c + W - 1 of the load,
//           W = TPL / 4.
//   values  the tokens a lane holds scores for are its 8 places of the sum, so
//           the weights go into the second operand as they are.  The first
//           operand wants 8 tokens' values of one d in a lane: lane (p, c)
//           loads values J p .. J p + J - 1 (J = D / 16) of those 8 tokens, an
//           8 x J matrix that it transposes in registers with byte permutes.
//           Tile j is then d = J p + j, and lane (n, c) ends with d = J (4 c +
//           v) + j, J values side by side.
// A 4-bit row is 64 bytes and its scales 4: lanes load a piece's scale beside it
// and convert to bf16 in registers, exactly.
// The weights enter as two bf16 terms (value and rest), so an output carries
// about 16 bits of them; the matrix units are idle either way.
//
// The running maximum moves only when a tile exceeds it by 2^8 (every weight is
// then at most 2^8, exact in float32 sums), so most tiles need no exchange
// between lanes.
//
// Measured, 8 kv heads of 128 with 4 queries each: 131072 bf16 tokens of one
// sequence with block sums (537 MB) 96 us, 5.6 TB/s; 64 e4m3 sequences of up to
// 32768 tokens (2.7 GB) 440 us, 6.1 TB/s, 256 of up to 8192 449 us, where nothing
// but streaming reads reaches 7.1.  About 18 us of a call are its start (lengths,
// table, first tiles) and end: 1024 tokens of one head of 64 take 8.0 us.  17 to
// 32 queries are two groups: 131072 tokens with 32 queries a head take 142 us and
// move 771 MB, with 16 queries 95 us and 538 MB (up to 15% more by where the cache lies
// in memory).  4-bit caches: 131072 tokens (143
// MB) 41 us, 64 sequences of up to 32768 (1.45 GB) 287, 5.1 TB/s; with a window of
// 4096 183 us in bf16 (1.07 GB, 5.8 TB/s), 107 in e4m3, 65 in 4 bits.  Loads and
// softmax without the products take 254 of the 287 us: pages of 1 KiB a head and
// their scales 64 bytes at a time are what bounds it.  Tried on it and not kept: two
// or three tiles ahead (39 us for 42, but 325 to 350 for 287), values turned by LDS
// transpose reads (314), loads of masked tiles too (bf16 97 -> 100), addresses from a
// scalar base (no change), three or four waves a SIMD (no change, spills).
template <int D, Held HELD>
struct StreamLayout {
    static constexpr int RB = (int)(HELD == FP4 ? D / 2 : (HELD == FP8 ? D : 2 * D));       // bytes of a row
    static constexpr int TPL = 1024 / RB;           // tokens of a wave-load
    static constexpr int NK = 32 / TPL;             // key loads of a tile
    static constexpr int W = TPL / 4;               // tokens a lane scores per load
    static constexpr int H = RB / 64;               // 64-byte parts of a row
    static constexpr int KP = HELD == FP4 ? 4 : (HELD == FP8 ? 2 : 1);      // products of 32 values per part
    static constexpr int J = D / 16;                // values a lane holds of a token
    static constexpr int VW = RB / 64;              // 4-byte words of them as stored
    static_assert(H >= 1, "a token's head fills a lane group");
};

// max / sum over the four lanes (n, 0..3) of a query
__device__ inline float max_over_c(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float sum_over_c(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The blocks of one sequence as a wave walks it: 64 blocks at a time, a lane
// each holding where its block lies (bytes from the head's start of the cache).
// Entries that are invalid, or of blocks the sequence does not use, stand for
// block 0: every address is inside the cache, and what is loaded there is masked.
template <bool WINDOW>
struct TableWindow {
    const int32_t* row;     // null: the identity
    int used, first;
    uint32_t lo, hi;
    uint64_t bad;           // used blocks with an invalid entry
    int unseen, unseen_end; // blocks that a window leaves out, whose entries may be anything

    __device__ inline void load(const AttendArgs& a, int block, int64_t block_bytes, int lane) {
        first = block;
        int e = 0;
        if (block + lane < used) e = row ? row[block + lane] : block + lane;
        const bool invalid = e < 0 || e >= a.N;
        bad = __ballot(invalid);
        if (WINDOW ? __ballot(invalid && !(block + lane >= unseen && block + lane < unseen_end)) != 0 && lane == 0
                   : bad && lane == 0)
            atomicOr(a.err, DEVERR_TABLE);
        const int64_t at = invalid ? 0 : e * block_bytes;
        lo = (uint32_t)at;
        hi = (uint32_t)(at >> 32);
    }
    // uniform; any index gives an address inside the cache
    __device__ inline int64_t at(int index) const {
        return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, index & 63) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)lo, index & 63));
    }
};

// What rows `from` (to `end`, by default the last) of a kv head get that have no
// live row in their group:
// block_lse -inf for this run's blocks and, where no join follows, output 0
// and lse -inf.
__device__ inline void write_dead_rows(const AttendArgs& a, const Item& it, const BlockSize& bs, int from, int t0, int t1,
                                       int end = 0x7FFFFFFF) {
    const int g = a.Hq / a.Hk, dead = (a.M * g < end ? a.M * g : end) - from;
    if (dead <= 0) return;
    if (a.block_lse && t1 > t0) {
        const int b0 = bs.block(t0), blocks = bs.block(t1 - 1) + 1 - b0;
        for (int64_t x = threadIdx.x; x < (int64_t)blocks * dead; x += 256) {
            const int r = from + (int)(x % dead), b = b0 + (int)(x / dead);
            a.block_lse[(((int64_t)it.s * a.n + b) * a.M + r / g) * a.Hq + it.kvh * g + r % g] = -INFINITY;
        }
    }
    if (it.share.runs > 1) return;
    for (int x = threadIdx.x; x < dead * (a.D / 8); x += 256) {
        const int r = from + x / (a.D / 8), d = x % (a.D / 8) * 8;
        const int64_t row = ((int64_t)it.s * a.M + r / g) * a.Hq + it.kvh * g + r % g;
        *reinterpret_cast<u32x4_t*>(a.out + row * a.D + d) = u32x4_t{0, 0, 0, 0};
        if (a.lse && d == 0) a.lse[row] = -INFINITY;
    }
}

// BYTES from a uniform address and a lane's offset, nontemporal (each byte is
// read once by a group of 16 queries).
template <int BYTES>
__device__ inline void stream_load(uint32_t* dst, const char* base, uint32_t off) {
    if constexpr (BYTES == 16) {
        const u32x4_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(base + off));
        dst[0] = x[0];
        dst[1] = x[1];
        dst[2] = x[2];
        dst[3] = x[3];
    } else if constexpr (BYTES == 8) {
        typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
        const u32x2_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(base + off));
        dst[0] = x[0];
        dst[1] = x[1];
    } else {
        dst[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(base + off));
    }
}

// A sequence's work where a window limits it.
struct WindowWork {
    static constexpr bool kChunk = false;
    const AttendArgs& a;
    __device__ inline void operator()(int s, int& len, int& groups) const {
        const int tokens = kv_len_of(a.kv_len, s, (int64_t)a.n * a.B), drafted = draft_len_of(a, s, tokens);
        len = span_of(a, tokens, drafted, 0, drafted - 1, 32).end;
        groups = 1;
    }
};

template <int D, Held HELD, bool WINDOW>
__global__ __launch_bounds__(256, 2) void attend_stream_kernel(AttendArgs a, Plan pl, BlockSize bs) {
    using L = StreamLayout<D, HELD>;
    constexpr int NK = L::NK, W = L::W, H = L::H, KP = L::KP, J = L::J, TPL = L::TPL, VW = L::VW;
    __shared__ float exchange[2][(J * 4 + 2) * 64];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, c = lane >> 4;
    Item it;
    if constexpr (WINDOW) it = item_of(a, pl, blockIdx.x, WindowWork{a});
    else it = item_of(a, pl, blockIdx.x, DraftWork{a, pl});
    if (it.slot < 0) return;
    if constexpr (WINDOW) it.share.len = kv_len_of(a.kv_len, it.s, (int64_t)a.n * a.B);
    const int s = it.s, kvh = it.kvh, len = it.share.len, drafted = draft_len_of(a, s, len);
    // t0, t1 and what counts tiles are places of the walk, which with a window leaves tokens out
    const Span span = WINDOW ? span_of(a, len, drafted, 0, drafted - 1, 32) : Span{len, 0, len};
    if (kvh == 0 && it.group == 0 && it.split == 0 && threadIdx.x == 0) {
        check_lengths(a, s, len, drafted);
        if (a.ws) shares_of(a)[s] = it.share;
    }
    const int ctx = len - drafted, t0 = it.split * it.share.run;
    const int t1 = t0 + it.share.run < span.end ? t0 + it.share.run : span.end;
    const int end = WINDOW ? span.real_end(t1) : t1;
    auto real = [&](int v) { return WINDOW ? span.real(v) : v; };
    const int g = a.Hq / a.Hk, R = a.M * g;

    if (!WINDOW && it.last) write_dead_rows(a, it, bs, 16 * (it.group + 1), t0, t1);

    // the lane's row, and the queries as second operands
    const int r = 16 * it.group + n, i = r / g;
    const bool live = r < R && i < drafted;
    const uint64_t seen = live && !WINDOW ? tree_word(a, s, i) : 0;
    const int pos = ctx + i, first = pos - a.window + 1;       // with a window
    auto sees_token = [&](int tok) {
        if constexpr (WINDOW) return tok <= pos && (tok >= first || tok < a.sinks);
        else return tok < ctx || ((seen >> ((tok - ctx) & 63)) & 1);
    };
    const int64_t row = ((int64_t)s * a.M + i) * a.Hq + kvh * g + r % g;
    const int64_t block_step = (int64_t)a.M * a.Hq;
    // where lane group c writes the c-th block of a tile that starts with block 0
    float* const block_row =
        a.block_lse ? a.block_lse + (((int64_t)s * a.n + (bs.B < 32 ? c : 0)) * a.M + i) * a.Hq + kvh * g + r % g : nullptr;
    bf16x8_t q[H][KP];
#pragma unroll
    for (int j = 0; j < H; ++j)
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            // a row that is not live weighs nothing: zeros, whatever it holds
            q[j][k] = bf16x8_t{};
            if (live) q[j][k] = signed_by(a.scale, load8(a.q + row * D + 8 * KP * (4 * j + c) + 8 * k));
        }

    const int ts = (int)bytes_of<HELD>(a.cache.token_stride), block_ts = bs.B * ts;
    const int64_t block_bytes = bytes_of<HELD>(a.cache.block_stride), head_off = bytes_of<HELD>(kvh * a.cache.head_stride);
    const char* const kp = static_cast<const char*>(a.cache.k) + head_off;
    const char* const vp = static_cast<const char*>(a.cache.v) + head_off;
    const uint32_t k_off = n / H * ts + 16 * (4 * (n % H) + c);
    uint32_t v_off[W];
#pragma unroll
    for (int w = 0; w < W; ++w) v_off[w] = (W * c + w) * ts + n * (VW * 4);
    // of a 4-bit cache: 16 bytes of values have a scale byte
    const uint8_t* const ksp = HELD == FP4 ? a.cache.k_scales + head_off / 16 : nullptr;
    const uint8_t* const vsp = HELD == FP4 ? a.cache.v_scales + head_off / 16 : nullptr;

    TableWindow<WINDOW> table;
    table.row = a.tables ? a.tables + (int64_t)s * a.n : nullptr;
    table.used = end > 0 ? bs.block(end - 1) + 1 : 0;
    table.unseen = table.unseen_end = 0;
    if constexpr (WINDOW) {
        const int lowest = ctx - a.window + 1;      // the first row's window
        table.unseen = bs.block(a.sinks + bs.B - 1);
        table.unseen_end = lowest > 0 ? bs.block(lowest) : 0;
    }

    // this wave's tiles: groups of `per` consecutive ones, every fourth group
    const int per = pl.unit / 128;
    auto tile_of = [&](int k) { return per == 1 ? t0 + 32 * (4 * k + wave) : t0 + 32 * ((k / per * 4 + wave) * per + k % per); };

    // Where a tile's wave-loads begin (each inside one block), moving the window if the tile is past it.
    int64_t place[NK];
    uint32_t kr[NK][4], vr[8][VW];
    uint32_t k_sc[NK], v_sc[8];     // their scale bytes
    auto places = [&](int t) {
        const int b = bs.block(t), last = bs.block(t + 31 < end ? t + 31 : end - 1);
        if (last >= table.first + 64) table.load(a, b, block_bytes, lane);
        int index = b - table.first, off = (t - b * bs.B) * ts;
#pragma unroll
        for (int u = 0; u < NK; ++u) {
            place[u] = table.at(index) + off;
            off += TPL * ts;
            const bool over = off == block_ts;
            off = over ? 0 : off;
            index += over;
        }
    };
    auto load_k = [&]() {
#pragma unroll
        for (int u = 0; u < NK; ++u) {
            stream_load<16>(kr[u], kp + place[u], k_off);
            if constexpr (HELD == FP4) k_sc[u] = (ksp + (place[u] >> 4))[k_off / 16];
        }
    };
    auto load_v = [&]() {
#pragma unroll
        for (int u = 0; u < NK; ++u)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                stream_load<VW * 4>(vr[u * W + w], vp + place[u], v_off[w]);
                if constexpr (HELD == FP4) v_sc[u * W + w] = (vsp + (place[u] >> 4))[v_off[w] / 16];
            }
    };

    f32x4_t o[J];
#pragma unroll
    for (int j = 0; j < J; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = kLowest, l = 0.f;
    float wide_m = kLowest, wide_l = 0.f;       // block_lse of a block wider than a tile: its maximum and sum so far
    const float scale = log2_scale(a);      // the queries carry its sign

    bool odd = false;       // a drafted token's value is not finite
    int at_tile = tile_of(0), t = real(at_tile);
    if (at_tile < t1) {
        table.load(a, bs.block(t), block_bytes, lane);
        places(t);
        load_k();
        load_v();
    }
    for (int k = 0; at_tile < t1; ++k) {
        const int next_tile = tile_of(k + 1), next = real(next_tile);
        // scores of this tile's 32 tokens
        float x[8];
#pragma unroll
        for (int u = 0; u < NK; ++u) {
            bf16x8_t key[KP];
            if constexpr (HELD == FP4) {
#pragma unroll
                for (int kk = 0; kk < KP; ++kk) key[kk] = __builtin_bit_cast(bf16x8_t, fp4x8_to_bf16(kr[u][kk], k_sc[u]));
            } else if constexpr (HELD == FP8) {
                key[0] = __builtin_bit_cast(bf16x8_t, (u32x4_t){fp8x2_to_bf16<false>(kr[u][0]), fp8x2_to_bf16<true>(kr[u][0]),
                                                                fp8x2_to_bf16<false>(kr[u][1]), fp8x2_to_bf16<true>(kr[u][1])});
                key[KP - 1] = __builtin_bit_cast(bf16x8_t, (u32x4_t){fp8x2_to_bf16<false>(kr[u][2]), fp8x2_to_bf16<true>(kr[u][2]),
                                                                     fp8x2_to_bf16<false>(kr[u][3]), fp8x2_to_bf16<true>(kr[u][3])});
            } else {
                key[0] = __builtin_bit_cast(bf16x8_t, (u32x4_t){kr[u][0], kr[u][1], kr[u][2], kr[u][3]});
            }
            f32x4_t part[H];
#pragma unroll
            for (int j = 0; j < H; ++j) {
                part[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < KP; ++kk)
                    part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key[kk], q[j][kk], part[j], 0, 0, 0);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                float sum = part[0][w * H];
#pragma unroll
                for (int j = 1; j < H; ++j) sum += part[j][w * H + j];
                x[u * W + w] = sum;
            }
        }
        // which loads of this tile lie in a block with an invalid entry (before the window moves on)
        uint32_t dead = 0;
        if (table.bad) {
#pragma unroll
            for (int u = 0; u < NK; ++u)
                dead |= (uint32_t)((table.bad >> ((bs.block(t + TPL * u) - table.first) & 63)) & 1) << u;
        }
        // (the last row's window begins at len - window)
        const bool masked = t + 32 > ctx || t + 32 > end || dead != 0 || (WINDOW && t < len - a.window && t + 32 > a.sinks);
        if (next_tile < t1) {
            places(next);
            load_k();
        }

        if (masked) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int u = e / W, tok = t + TPL * u + W * c + e % W;
                const bool there = tok < end && !((dead >> u) & 1);
                const bool some = WINDOW || tok >= ctx;         // perhaps not every row sees it
                const bool sees = there && sees_token(tok);
                x[e] = sees ? x[e] : -INFINITY;
                if constexpr (HELD == FP4) {
                    const bool bad = v_sc[e] == 255u;
                    odd |= bad && there && some;
                    if (!there || (bad && some)) vr[e][0] = v_sc[e] = 0u;
                } else {
#pragma unroll
                    for (int y = 0; y < VW; ++y) {
                        vr[e][y] = there ? vr[e][y] : 0u;       // no value there at all
                        const uint32_t finite = HELD == FP8 ? finite_only_fp8(vr[e][y]) : finite_only(vr[e][y]);
                        if (some && finite != vr[e][y]) {
                            vr[e][y] = finite;
                            odd = true;
                        }
                    }
                }
            }
        }

        // the running maximum, in log2 units; weights 2^(score - maximum)
        float top[4];       // of each pair of places
#pragma unroll
        for (int y = 0; y < 4; ++y) top[y] = max3(kLowest, x[2 * y], x[2 * y + 1]);
        const float tile_top = max3(max3(top[0], top[1], top[2]), top[3], kLowest) * scale;
        if (__ballot(tile_top > m + 8.f)) {
            const float m_new = fmaxf(m, max_over_c(tile_top));
            const float alpha = exp2_of(m - m_new);
            m = m_new;
            l *= alpha;
#pragma unroll
            for (int j = 0; j < J; ++j) o[j] *= alpha;
        }
        if (!WINDOW && a.block_lse) {
            // Blocks of 8 or 16 tokens lie side by side in a tile, in 2 or 4 of a lane's 8 places; one of 32 or more
            // fills it.  Their sums are those of the weights, brought back by the maximum, unless one lies so far
            // below it that its weights are lost: then the sums are taken against each block's own maximum.
            auto blocks = [&](auto parts_) {
                constexpr int parts = decltype(parts_)::value, each = 8 / parts;
                float part_top[parts], sum[parts], ref[parts];
                bool far = false;
#pragma unroll
                for (int y = 0; y < parts; ++y) {
                    part_top[y] = top[y * each / 2];
#pragma unroll
                    for (int e = 1; e < each / 2; ++e) part_top[y] = fmaxf(part_top[y], top[y * each / 2 + e]);
                    far |= part_top[y] * scale < m - 60.f && part_top[y] > kLowest;
                    sum[y] = 0.f;
                    ref[y] = m;
                }
                const bool own = __ballot(far) != 0;
                if (own) {
#pragma unroll
                    for (int y = 0; y < parts; ++y) {
                        ref[y] = fmaxf(max_over_c(part_top[y]) * scale, kLowest);
#pragma unroll
                        for (int e = 0; e < each; ++e) sum[y] += exp2_of(__builtin_fmaf(x[y * each + e], scale, -ref[y]));
                    }
                }
#pragma unroll
                for (int y = 0; y < parts; ++y) {
                    float part_l = 0.f;
#pragma unroll
                    for (int e = 0; e < each; ++e) {
                        x[y * each + e] = exp2_of(__builtin_fmaf(x[y * each + e], scale, -m));
                        part_l += x[y * each + e];
                    }
                    l += part_l;
                    sum[y] = sum_over_c(own ? sum[y] : part_l);
                }
                float mine_sum = sum[0], mine_ref = ref[0];
#pragma unroll
                for (int y = 1; y < parts; ++y) {
                    mine_sum = y == c ? sum[y] : mine_sum;
                    mine_ref = y == c ? ref[y] : mine_ref;
                }
                if constexpr (parts == 1) {
                    // a tile in which the row sees nothing is taken against the running maximum: it counts for nothing, and
                    // must not raise the block's reference, from which the sum so far may lie too far to be held
                    if (mine_sum == 0.f) mine_ref = kLowest;
                    const float both = fmaxf(wide_m, mine_ref);
                    wide_l = wide_l * exp2_of(wide_m - both) + mine_sum * exp2_of(mine_ref - both);
                    wide_m = both;
                    mine_sum = wide_l;
                    mine_ref = both;
                }
                const int b = bs.block(t);
                // of a block wider than a tile: with its last tile, or the sequence's
                const bool done = parts > 1 || t + 32 >= t1 || bs.block(t + 32) != b;
                if (done && c < parts && r < R && t + 32 / parts * c < t1)
                    block_row[(int64_t)b * block_step] =
                        live && !(mine_sum <= 0.f) ? (mine_ref + log2_of(mine_sum)) * kLn2 : -INFINITY;
                if (parts == 1 && done) {
                    wide_m = kLowest;
                    wide_l = 0.f;
                }
            };
            if (bs.B == 16) blocks(std::integral_constant<int, 2>());
            else if (bs.B == 8) blocks(std::integral_constant<int, 4>());
            else blocks(std::integral_constant<int, 1>());
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = exp2_of(__builtin_fmaf(x[e], scale, -m));
                l += x[e];
            }
        }

        u32x4_t wh, wl;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wh[e] = bf16_pair(x[2 * e], x[2 * e + 1]);
            wl[e] = bf16_pair(rest_of<false>(x[2 * e], wh[e]), rest_of<true>(x[2 * e + 1], wh[e]));
        }
        const bf16x8_t hi = __builtin_bit_cast(bf16x8_t, wh), lo = __builtin_bit_cast(bf16x8_t, wl);

        // values as bf16 words, J / 2 of each token
        uint32_t vw[8][J / 2];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (HELD == FP4) {
                const u32x4_t w = fp4x8_to_bf16(vr[e][0], v_sc[e]);
#pragma unroll
                for (int y = 0; y < 4; ++y) vw[e][y] = w[y];
            } else if constexpr (HELD == FP8) {
#pragma unroll
                for (int y = 0; y < VW; ++y) {
                    vw[e][2 * y] = fp8x2_to_bf16<false>(vr[e][y]);
                    vw[e][2 * y + 1] = fp8x2_to_bf16<true>(vr[e][y]);
                }
            } else {
#pragma unroll
                for (int y = 0; y < VW; ++y) vw[e][y] = vr[e][y];
            }
        }
        // first operand of d = J p + j: that value of the lane's 8 tokens
#pragma unroll
        for (int j = 0; j < J; ++j) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = __builtin_amdgcn_perm(vw[2 * e + 1][j / 2], vw[2 * e][j / 2], j % 2 ? 0x07060302 : 0x05040100);
            const bf16x8_t val = __builtin_bit_cast(bf16x8_t, w);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(val, hi, o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(val, lo, o[j], 0, 0, 0);
        }
        if (next_tile < t1) load_v();
        at_tile = next_tile;
        t = next;
    }

    l = sum_over_c(l);
    bool lost = false;
    if constexpr (HELD == BF16) {
        float x = 0.f;      // NaN where a sum is not finite
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) x = __builtin_fmaf(o[j][v], 0.f, x);
        lost = x != 0.f && l == l;
    }
    const bool all = __ballot(lost) != 0;
    if (all || __ballot(odd)) {
        float sum[4][J];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int j = 0; j < J; ++j) sum[v][j] = 0.f;
        for (int v = all || WINDOW || ctx < t0 ? t0 : ctx; v < t1; ++v) {
            if ((v - t0) / 32 / per % 4 != wave) continue;          // another wave's
            const int tok = real(v);
            const char* const from = value_row<HELD>(a, bs, s, kvh, tok);
            if (from && sees_token(tok)) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int j = 0; j < J; j += 4) add_not_finite<HELD>(sum[v] + j, from, J * (4 * c + v) + j);
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int j = 0; j < J; ++j) o[j][v] = sum[v][j] == 0.f ? o[j][v] : sum[v][j];
    }

    // the waves' sums: 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
    for (int round = 2; round >= 1; round >>= 1) {
        if (wave >= round && wave < 2 * round) {
            float* const to = exchange[wave - round];
            to[4 * J * 64 + lane] = m;
            to[(4 * J + 1) * 64 + lane] = l;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) to[(4 * j + v) * 64 + lane] = o[j][v];
        }
        __syncthreads();
        if (wave < round) {
            const float* const from = exchange[wave];
            const float m_other = from[4 * J * 64 + lane], m_new = fmaxf(m, m_other);
            const float f = exp2_of(m - m_new), f_other = exp2_of(m_other - m_new);
            l = l * f + from[(4 * J + 1) * 64 + lane] * f_other;
            m = m_new;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) o[j][v] = joined(o[j][v], f, from[(4 * j + v) * 64 + lane], f_other);
        }
        __syncthreads();
    }
    if (wave != 0 || r >= R) return;
    const bool none = !live || l == 0.f;
    if (it.share.runs == 1) {       // the result
        const float f = none ? 0.f : a.cache.v_scale / l;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            uint32_t w[J / 2];
#pragma unroll
            for (int y = 0; y < J / 2; ++y) w[y] = none ? 0u : bf16_pair(o[2 * y][v] * f, o[2 * y + 1][v] * f);
            uint32_t* const to = reinterpret_cast<uint32_t*>(a.out + row * D + J * (4 * c + v));
#pragma unroll
            for (int y = 0; y < J / 2; ++y) to[y] = w[y];
        }
        if (a.lse && c == 0) a.lse[row] = none ? -INFINITY : (m + log2_of(l)) * kLn2;
    } else if (live) {
        float* const to = part_sums(a, pl, it.slot) + n * D;
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int y = 0; y < J / 4; ++y)
                *reinterpret_cast<float4*>(to + J * (4 * c + v) + 4 * y) =
                    make_float4(o[4 * y][v], o[4 * y + 1][v], o[4 * y + 2][v], o[4 * y + 3][v]);
        if (c == 0) part_stats(a, pl, it.slot)[n] = make_float2(m, l);
    }
}

// ---------------------------------------------------------------- tree kernel
//
// More than 32 queries per kv head (a draft tree), and the block sizes that the
// stream kernel does not take: a workgroup's four waves share tiles of 64
// tokens, staged through LDS as bf16 (an FP8 cache is converted on the way),
// each wave with 32 queries of its own, or, in a group of up to 64 live ones,
// two waves with the same 32 queries and half of each tile each (`pairs`).  The
// stage is double buffered: a tile's loads are issued before the previous tile
// is computed.  A bf16 tile of the context goes straight into LDS (64 full rows:
// 991 us a call through registers, 930 without); e4m3 is converted in
// registers on the way, and tiles with drafted or missing tokens are cleaned
// there.
//
// Both products run on v_mfma_f32_32x32x16_bf16 with the queries as the second
// operand, so lane (n = lane % 32, f = lane / 32) owns query n: it holds the
// scores of tokens v % 4 + 8 (v / 4) + 4 f, v = 0 .. 15, of 32, and its 16
// weights go into the second operand of the value product as they stand, 8 to
// a product.  The first operand of that product wants, for the same tokens, 4
// consecutive tokens' values of one d in a lane: the LDS transpose read gives a
// group of 16 lanes the 4 x 16 block whose rows its lanes point at.  A softmax
// reduction crosses lanes once (n and n + 32).
//
// LDS rows are 2 D bytes without padding; their 16-byte pieces are permuted by
// the row so that the 16 rows of a key read, and the 4 rows of a transpose read,
// fall on different banks.
//
// Bound: a tile's products, exponentials and LDS reads follow one another in each
// wave, with two waves a SIMD (the registers' limit), so the matrix cores idle for
// more than half of the time (the cache's bytes would take a quarter of it); the
// weights' second bf16 term makes the value product twice as long.  Measured, 16
// sequences of 16384 tokens, 64 rows of 8 queries for each of 8 heads of 128: 891
// us, 617 TFLOP/s (a matrix product of the library's reaches 1233), the matrix
// cores busy in 46% of the SIMDs' cycles; with block sums and lengths and drafts
// that vary 484 us (458 from an e4m3 cache), 24%.  13 rows over 8 sequences of 5k
// tokens: 58 us (50), 16%: an item's start and a chain of 10 to 12 tiles.
// BLOCKS: block sums a half tile has: 0 without block_lse, 1 for blocks of 32
// tokens or more, 2 for 16, 4 for 8.
template <int D, Held HELD, int BLOCKS>
__global__ __launch_bounds__(256, 2) void attend_tree_kernel(AttendArgs a, Plan pl, BlockSize bs) {
    using T = TreeLds<D>;
    constexpr int RB = (int)(HELD == FP4 ? D / 2 : (HELD == FP8 ? D : 2 * D));      // bytes of a cache row
    constexpr int CR = RB / 16;                 // 16-byte pieces of it
    constexpr int NR = (64 * CR + 255) / 256;   // pieces a thread stages, of keys and of values
    constexpr int SPREAD = 2 * D / RB;          // pieces of an LDS row that one becomes
    constexpr int KS = D / 16, DT = D / 32;
    __shared__ __attribute__((aligned(16))) char lds[4 * T::kTile];     // keys 0, keys 1, values 0, values 1
    __shared__ int any_odd;         // a drafted token's value is not finite

    const Item it = item_of(a, pl, blockIdx.x, DraftWork{a, pl});
    if (it.slot < 0) return;
    const int s = it.s, kvh = it.kvh, len = it.share.len, drafted = draft_len_of(a, s, len);
    if (kvh == 0 && it.group == 0 && it.split == 0 && threadIdx.x == 0) {
        check_lengths(a, s, len, drafted);
        if (a.ws) shares_of(a)[s] = it.share;
    }
    const int ctx = len - drafted, t0 = it.split * it.share.run;
    const int t1 = t0 + it.share.run < len ? t0 + it.share.run : len;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, f = lane >> 5;
    const int g = a.Hq / a.Hk, R = a.M * g;
    if (it.last) write_dead_rows(a, it, bs, 128 * (it.group + 1), t0, t1);
    // up to 64 live queries: two waves each, a half of every tile (not where a block's sum spans the halves)
    const bool pairs = drafted * g - 128 * it.group <= 64 && !(BLOCKS == 1 && bs.B > 32);
    if (pairs && it.last) write_dead_rows(a, it, bs, 128 * it.group + 64, t0, t1, 128 * (it.group + 1));
    const int in_group = (pairs ? wave / 2 : wave) * 32, r0 = 128 * it.group + in_group, r = r0 + n, i = r / g;
    const bool live = r < R && i < drafted;
    const bool wave_live = r0 < R && r0 / g < drafted;          // rows of a wave die from the end
    const uint64_t seen = live ? tree_word(a, s, i) : 0;
    // where lane f writes the f-th block of a half tile that starts with block 0
    float* const block_row =
        a.block_lse ? a.block_lse + (((int64_t)s * a.n + (bs.B < 32 ? f : 0)) * a.M + i) * a.Hq + kvh * g + r % g : nullptr;
    const int64_t block_step = (int64_t)a.M * a.Hq;
    const int64_t row = ((int64_t)s * a.M + i) * a.Hq + kvh * g + r % g;

    bf16x8_t q[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        q[k] = bf16x8_t{};
        if (live) q[k] = signed_by(a.scale, load8(a.q + row * D + 16 * k + 8 * f));
    }

    const int64_t head_off = bytes_of<HELD>(kvh * a.cache.head_stride);
    const char* const kp = static_cast<const char*>(a.cache.k) + head_off;
    const char* const vp = static_cast<const char*>(a.cache.v) + head_off;
    const int32_t* const table = a.tables ? a.tables + (int64_t)s * a.n : nullptr;

    // Staging.  Lane x of every wave finds where token x of a tile lies (bytes from the head's start; 0 and a bit in
    // `nowhere` for a token past the run's end or in a block with an invalid entry), and the threads take the offsets
    // of the tokens whose pieces they stage from there.
    auto entry_of = [&](int t) {
        const int tok = t + lane;
        if (tok >= t1) return -1;
        const int b = bs.block(tok);
        return table ? table[b] : b;
    };
    auto offset_of = [&](int t, int slot, uint64_t& nowhere) -> int64_t {
        const int tok = t + lane;
        const bool none = tok >= t1 || slot < 0 || slot >= a.N;
        nowhere = __ballot(none);
        return none ? 0 : bytes_of<HELD>(slot * a.cache.block_stride + (int64_t)(tok - bs.block(tok) * bs.B) * a.cache.token_stride);
    };
    const int my_tok = threadIdx.x / CR, my_piece = threadIdx.x % CR;     // and tokens 256 / CR further on
    const bool mine_in = 256 / CR * NR <= 64 || my_tok < 64;     // (64 values in 4 bits: half of the threads have a piece)
    u32x4_t ks[NR], vs[NR];
    uint32_t k_sc[NR], v_sc[NR];        // a piece's scale byte
    auto load_tile = [&](int64_t off) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int from = my_tok + 256 / CR * x;
            const int64_t o = ((int64_t)__shfl((int)(off >> 32), from) << 32 | (uint32_t)__shfl((int)off, from)) +
                              16 * my_piece;
            ks[x] = *reinterpret_cast<const u32x4_t*>(kp + o);
            vs[x] = *reinterpret_cast<const u32x4_t*>(vp + o);
            if constexpr (HELD == FP4) {
                k_sc[x] = a.cache.k_scales[(head_off + o) >> 4];
                v_sc[x] = a.cache.v_scales[(head_off + o) >> 4];
            }
        }
    };
    // 256 / CR is a multiple of 16, so a thread's rows share their permutation and lie a fixed step apart
    const int turn = HELD == FP4 ? my_tok & (SPREAD - 1) : 0;       // of a thread's values: see turned()
    const int k_to = T::key(my_tok, SPREAD * my_piece), v_to = T::value(my_tok, SPREAD * my_piece) ^ (16 * turn);
    auto store_tile = [&](int buf, int t, uint64_t nowhere) {
        if (!mine_in) return;
        if (t + 64 > ctx || nowhere != 0) {
            bool odd = false;
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const int tok = my_tok + 256 / CR * x;
                const bool none = (nowhere >> tok) & 1, tail = t + tok >= ctx;
                if constexpr (HELD == FP4) {
                    const bool bad = v_sc[x] == 255u;
                    odd |= bad && tail && !none;
                    if (none || (bad && tail)) {
                        vs[x] = u32x4_t{0, 0, 0, 0};
                        v_sc[x] = 0;
                    }
                }
#pragma unroll
                for (int y = 0; y < 4 && HELD != FP4; ++y) {
                    const uint32_t w = none ? 0u : vs[x][y];
                    const uint32_t finite = HELD == FP8 ? finite_only_fp8(w) : finite_only(w);
                    odd |= tail && finite != w;
                    vs[x][y] = tail ? finite : w;
                }
            }
            if (odd) any_odd = 1;
        }
        char* const kt = lds + buf * T::kTile + k_to;
        char* const vt = lds + (2 + buf) * T::kTile + v_to;
        if constexpr (HELD == FP4) {
#pragma unroll
            for (int x = 0; x < NR; ++x) vs[x] = turned(vs[x], turn);
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            constexpr int kStep = 256 / CR * T::kRow;
            if constexpr (HELD == FP4) {
                // the piece's quarters are pieces 4 p .. 4 p + 3: as below
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    *reinterpret_cast<u32x4_t*>(lds + buf * T::kTile + (k_to ^ (16 * y)) + x * kStep) = fp4x8_to_bf16(ks[x][y], k_sc[x]);
                    *reinterpret_cast<u32x4_t*>(lds + (2 + buf) * T::kTile + (v_to ^ (16 * y)) + x * kStep) = fp4x8_to_bf16(vs[x][y], v_sc[x]);
                }
            } else if constexpr (HELD == FP8) {
                // the piece's two halves are pieces 2 p and 2 p + 1: the permutation flips at most their last bit
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    u32x4_t wk, wv;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        wk[2 * z] = fp8x2_to_bf16<false>(ks[x][2 * y + z]);
                        wk[2 * z + 1] = fp8x2_to_bf16<true>(ks[x][2 * y + z]);
                        wv[2 * z] = fp8x2_to_bf16<false>(vs[x][2 * y + z]);
                        wv[2 * z + 1] = fp8x2_to_bf16<true>(vs[x][2 * y + z]);
                    }
                    *reinterpret_cast<u32x4_t*>(lds + buf * T::kTile + (k_to ^ (16 * y)) + x * kStep) = wk;
                    *reinterpret_cast<u32x4_t*>(lds + (2 + buf) * T::kTile + (v_to ^ (16 * y)) + x * kStep) = wv;
                }
            } else {
                *reinterpret_cast<u32x4_t*>(kt + x * kStep) = ks[x];
                *reinterpret_cast<u32x4_t*>(vt + x * kStep) = vs[x];
            }
        }
    };
    // Straight into LDS, where the bytes go as they are: a wave's 1 KiB lies there in the order of its lanes, so each
    // lane fetches the piece that belongs in its place.
    const int k_piece = my_piece ^ (D == 128 ? my_tok & 15 : (my_tok >> 1) & 7);
    const int v_piece = my_piece ^ (D == 128 ? (my_tok & 3) * 4 : ((my_tok >> 1) & 1) * 4);
    const uint32_t lds_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds +
                                                           wave * (64 / CR) * T::kRow);
    auto direct_load = [&](uint32_t to, const char* from) {
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)from,
                                         (__attribute__((address_space(3))) uint32_t*)to, 16, 0, 0);
    };
    auto direct_tile = [&](int buf, int64_t off) {
        int64_t at[NR];
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int from = my_tok + 256 / CR * x;
            at[x] = (int64_t)__shfl((int)(off >> 32), from) << 32 | (uint32_t)__shfl((int)off, from);
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const uint32_t to = lds_at + buf * T::kTile + 256 / CR * x * T::kRow;
            direct_load(to, kp + at[x] + 16 * k_piece);
            direct_load(to + 2 * T::kTile, vp + at[x] + 16 * v_piece);
        }
    };
    // A lane's reads: key row n, piece 2 k + f; value row 4 f + l16 / 4, column 32 d + 16 * (lane / 16 % 2) + 4 * (l16 %
    // 4).  Rows a multiple of 16 (keys) or 4 (values) further on have the same permutation, and it is an exclusive or,
    // so k and d enter as one.
    const int l16 = lane & 15;
    const int k_from = T::key(n, f);
    const int v_from = T::value(4 * f + l16 / 4, 2 * ((lane >> 4) & 1) + l16 % 4 / 2) + 8 * (l16 % 2);

    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16_t{};
    float m = kLowest, l = 0.f, wide_m = kLowest, wide_l = 0.f;
    const float scale = log2_scale(a);

    if (threadIdx.x == 0) any_odd = 0;
    __syncthreads();
    uint64_t nowhere, nowhere_next = 0;
    int slot = entry_of(t0);
    load_tile(offset_of(t0, slot, nowhere));
    slot = entry_of(t0 + 64);
    store_tile(0, t0, nowhere);
    __syncthreads();
    // HALVES = 2: the whole of every tile; 1: half `mine` of it
    auto walk = [&](auto halves_, const int mine) {
        constexpr int HALVES = decltype(halves_)::value;
        for (int t = t0, buf = 0; t < t1; t += 64, buf ^= 1) {
            const bool more = t + 64 < t1;
            bool direct = false;        // no drafted tokens, none missing: nothing to look at
            int64_t off = 0;
            if (more) {
                off = offset_of(t + 64, slot, nowhere_next);
                direct = HELD == BF16 && t + 128 <= ctx && nowhere_next == 0;
                if (direct) direct_tile(buf ^ 1, off);
                else if (HELD != BF16) load_tile(off);
                slot = entry_of(t + 128);
            }
            uint64_t wrong = nowhere;       // invalid entries: tokens past the run's end are none
            if (t + 64 > t1) wrong &= (1ull << (t1 - t)) - 1;
            if (wrong && wave == 0 && lane == 0) atomicOr(a.err, DEVERR_TABLE);
            if (wave_live) {
                float x[HALVES][16];
                const char* const kt = lds + buf * T::kTile + (HALVES == 1 ? 32 * mine * T::kRow : 0);
                const char* const vt = kt + 2 * T::kTile;
                const int th = t + 32 * mine;
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    f32x16_t acc = f32x16_t{};
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const bf16x8_t key = __builtin_bit_cast(
                            bf16x8_t, *reinterpret_cast<const u32x4_t*>(kt + (k_from ^ (32 * k)) + 32 * h * T::kRow));
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key, q[k], acc, 0, 0, 0);
                    }
#pragma unroll
                    for (int v = 0; v < 16; ++v) x[h][v] = acc[v];
                }
                if (t + 64 > ctx || nowhere != 0) {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const uint32_t dead = (uint32_t)(nowhere >> (32 * (h + mine)));
#pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const int in = v % 4 + 8 * (v / 4) + 4 * f, place = th + 32 * h + in - ctx;
                            const bool sees = ((dead >> in) & 1) == 0 && (place < 0 || ((seen >> (place & 63)) & 1));
                            x[h][v] = sees ? x[h][v] : -INFINITY;
                        }
                    }
                }

                // the running maximum and the blocks' sums as in the stream kernel; 8-token blocks are quads of v,
                // 16-token ones pairs of quads
                float top[HALVES][4], tile_top = kLowest;
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        top[h][y] = max3(max3(kLowest, x[h][4 * y], x[h][4 * y + 1]), x[h][4 * y + 2], x[h][4 * y + 3]);
                        if (y % 2) tile_top = max3(tile_top, top[h][y - 1], top[h][y]);
                    }
                tile_top *= scale;
                if (__ballot(tile_top > m + 8.f)) {
                    const float m_new = fmaxf(m, max_over_f(tile_top));
                    const float alpha = exp2_of(m - m_new);
                    m = m_new;
                    l *= alpha;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= alpha;
                }
                constexpr int kSums = BLOCKS ? BLOCKS : 1, each = 16 / kSums;
                float sum[HALVES][kSums], ref[HALVES][kSums];
                bool own = false;
                if constexpr (BLOCKS > 0) {
                    bool far = false;
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
#pragma unroll
                        for (int b = 0; b < BLOCKS; ++b) {
                            float& part_top = ref[h][b];
                            part_top = top[h][b * each / 4];
#pragma unroll
                            for (int e = 1; e < each / 4; ++e) part_top = fmaxf(part_top, top[h][b * each / 4 + e]);
                            far |= part_top * scale < m - 60.f && part_top > kLowest;
                        }
                    own = __ballot(far) != 0;
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
#pragma unroll
                        for (int b = 0; b < BLOCKS; ++b) {
                            sum[h][b] = 0.f;
                            if (own) {
                                ref[h][b] = fmaxf(max_over_f(ref[h][b]) * scale, kLowest);
#pragma unroll
                                for (int e = 0; e < each; ++e)
                                    sum[h][b] += exp2_of(__builtin_fmaf(x[h][b * each + e], scale, -ref[h][b]));
                            } else {
                                ref[h][b] = m;
                            }
                        }
                }

#pragma unroll
                for (int h = 0; h < HALVES; ++h)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float* const w = x[h] + 8 * y;
                        float part_l[2] = {0.f, 0.f};       // of each quad
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            w[e] = exp2_of(__builtin_fmaf(w[e], scale, -m));
                            part_l[e / 4] += w[e];
                        }
                        l += part_l[0] + part_l[1];
                        if constexpr (BLOCKS > 0) {
                            if (!own) {
                                sum[h][8 * y / each] += part_l[0];
                                sum[h][(8 * y + 4) / each] += part_l[1];
                            }
                        }
                        u32x4_t wh, wl;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            wh[e] = bf16_pair(w[2 * e], w[2 * e + 1]);
                            wl[e] = bf16_pair(rest_of<false>(w[2 * e], wh[e]), rest_of<true>(w[2 * e + 1], wh[e]));
                        }
                        // 8 tokens' values of one d: two transpose reads
                        bf16x8_t val[DT];
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            struct { i16x4_t p[2]; } both;
#pragma unroll
                            for (int z = 0; z < 2; ++z)
                                both.p[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                    (lds_i16x4_t*)(vt + (v_from ^ (64 * d)) + (32 * h + 16 * y + 8 * z) * T::kRow));
                            val[d] = __builtin_bit_cast(bf16x8_t, both);
                        }
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(val[d], __builtin_bit_cast(bf16x8_t, wh), o[d], 0, 0, 0);
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(val[d], __builtin_bit_cast(bf16x8_t, wl), o[d], 0, 0, 0);
                    }

                if constexpr (BLOCKS > 0) {
                    // lane f writes blocks f, f + 2 of a half; a single one lane 0
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const int half = th + 32 * h, b = bs.block(half);
                        const bool done = BLOCKS > 1 || half + 32 >= t1 || bs.block(half + 32) != b;
                        if (half >= t1) break;
#pragma unroll
                        for (int y = 0; y < (BLOCKS + 1) / 2; ++y) {
                            float mine_sum = sum_over_f(sum[h][2 * y]), mine_ref = ref[h][2 * y];
                            if constexpr (BLOCKS > 1) {
                                const float other = sum_over_f(sum[h][2 * y + 1]);
                                mine_sum = f ? other : mine_sum;
                                mine_ref = f ? ref[h][2 * y + 1] : mine_ref;
                            } else {
                                if (mine_sum == 0.f) mine_ref = kLowest;        // as in the stream kernel
                                const float both = fmaxf(wide_m, mine_ref);
                                wide_l = wide_l * exp2_of(wide_m - both) + mine_sum * exp2_of(mine_ref - both);
                                wide_m = both;
                                mine_sum = wide_l;
                                mine_ref = both;
                            }
                            if (done && f < BLOCKS && r < R && half + 32 / BLOCKS * (2 * y + f) < t1)
                                block_row[(int64_t)(b + 2 * y) * block_step] =
                                    live && !(mine_sum <= 0.f) ? (mine_ref + log2_of(mine_sum)) * kLn2 : -INFINITY;
                        }
                        if (BLOCKS == 1 && done) {
                            wide_m = kLowest;
                            wide_l = 0.f;
                        }
                    }
                }
            } else if (BLOCKS > 0 && r < R && !(pairs && wave % 2)) {     // empty rows in a workgroup that has others
                const int last = bs.block(t + 63 < t1 ? t + 63 : t1 - 1);
                for (int b = bs.block(t); b + (bs.B < 32 ? f : 0) <= last; b += bs.B < 32 ? 2 : 1)
                    block_row[b * block_step] = -INFINITY;
            }
            if (direct) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // in LDS before the barrier
            } else if (more) {
                if (HELD == BF16) load_tile(off);
                store_tile(buf ^ 1, t + 64, nowhere_next);
            }
            nowhere = nowhere_next;
            __syncthreads();
        }
    };
    if (pairs) walk(std::integral_constant<int, 1>(), wave % 2);
    else walk(std::integral_constant<int, 2>(), 0);

    l = sum_over_f(l);
    bool lost = false;
    if constexpr (HELD == BF16) {
        float x = 0.f;      // NaN where a sum is not finite
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int v = 0; v < 16; ++v) x = __builtin_fmaf(o[d][v], 0.f, x);
        lost = x != 0.f && l == l;
    }
    const bool all = __ballot(lost) != 0;
    if (all || any_odd) {
        // 32 of a token's values at a time: the sums of them all would be too many registers beside o
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            float sum[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) sum[v] = 0.f;
            for (int tok = all || ctx < t0 ? t0 : ctx; tok < t1; ++tok) {
                if (pairs && (tok - t0) / 32 % 2 != wave % 2) continue;         // the other wave's half
                const char* const from = value_row<HELD>(a, bs, s, kvh, tok);
                if (from && (tok < ctx || ((seen >> ((tok - ctx) & 63)) & 1))) {
#pragma unroll
                    for (int v = 0; v < 16; v += 4) add_not_finite<HELD>(sum + v, from, 32 * d + 2 * v + 4 * f);
                }
            }
#pragma unroll
            for (int v = 0; v < 16; ++v) o[d][v] = sum[v] == 0.f ? o[d][v] : sum[v];
        }
    }
    if (pairs) {
        // the pair's sums, through the (now unused) stage
        float* const x = reinterpret_cast<float*>(lds) + (wave / 2) * (16 * DT + 2) * 64;
        if (wave % 2) {
            x[lane] = m;
            x[64 + lane] = l;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int v = 0; v < 16; ++v) x[(2 + 16 * d + v) * 64 + lane] = o[d][v];
        }
        __syncthreads();
        if (wave % 2) return;
        const float m_other = x[lane], m_new = fmaxf(m, m_other);
        const float mine = exp2_of(m - m_new), other = exp2_of(m_other - m_new);
        l = l * mine + x[64 + lane] * other;
        m = m_new;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[d][v] = joined(o[d][v], mine, x[(2 + 16 * d + v) * 64 + lane], other);
    }
    if (r >= R) return;
    const bool none = !live || l == 0.f;
    if (it.share.runs == 1) {
        const float inv = none ? 0.f : a.cache.v_scale / l;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint2 w = make_uint2(bf16_pair(o[d][4 * y] * inv, o[d][4 * y + 1] * inv),
                                     bf16_pair(o[d][4 * y + 2] * inv, o[d][4 * y + 3] * inv));
                if (none) w = make_uint2(0, 0);
                *reinterpret_cast<uint2*>(a.out + row * D + 32 * d + 8 * y + 4 * f) = w;
            }
        if (a.lse && f == 0) a.lse[row] = none ? -INFINITY : (m + log2_of(l)) * kLn2;
    } else if (live) {
        float* const to = part_sums(a, pl, it.slot) + (in_group + n) * D;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<float4*>(to + 32 * d + 8 * y + 4 * f) =
                    make_float4(o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2], o[d][4 * y + 3]);
        if (f == 0) part_stats(a, pl, it.slot)[in_group + n] = make_float2(m, l);
    }
}

// ---------------------------------------------------------------- choice of a kernel

enum class Kind { Stream, Tree, Plain, Chunk };

int queries_of(const AttendArgs& a) { return a.M * (a.Hq / a.Hk); }

constexpr int kRounds = 8;              // most workgroups a CU's places get one after another
// Queries per kv head of the stream kernel.  Two groups of 16 read most bytes twice: over 131072 tokens of one sequence
// 32 queries take 142 us with it, and 40 take 111 with the tree kernel; where they cross below 32 has not been measured.
constexpr int kStreamQueries = 32;
Kind kind_of(const AttendArgs& a) {
    const Held held = held_of(a.cache);
    auto bytes = [held](int64_t x) { return held == FP4 ? bytes_of<FP4>(x) : (held == FP8 ? bytes_of<FP8>(x) : bytes_of<BF16>(x)); };
    if (a.D != 64 && a.D != 128) return Kind::Plain;
    // a block's sum is taken inside a tile, or over whole tiles
    if (a.block_lse && (!(a.B % 32 == 0 || a.B == 16 || a.B == 8) || a.B > 65536)) return Kind::Plain;
    // 16-byte loads
    if (!aligned_to(a.cache.k, 16) || !aligned_to(a.cache.v, 16) ||
        bytes(a.cache.block_stride | a.cache.token_stride | a.cache.head_stride) % 16 != 0)
        return Kind::Plain;
    // the stream kernel's wave-loads take tokens of one block, all within 32-bit offsets of its first (the tree kernel
    // finds every token's place for itself, so it has the rest: 16 sequences of 8192 tokens of 64 e4m3 values in blocks
    // of 8 take 39 us with it, 2021 with the plain kernel)
    // a row of 64 values in 4 bits is 32 bytes, half of what the stream kernel's lane groups take
    const int tpl = (int)(1024 / bytes(a.D));
    const bool fits = a.B % tpl == 0 && a.cache.token_stride <= (1 << 24) &&
                      bytes(a.B * a.cache.token_stride) <= 0x7FFFFFFF && !(held == FP4 && a.D == 64);
    if (a.window) return fits && queries_of(a) <= kWindowQueries ? Kind::Stream : Kind::Chunk;
    return fits && queries_of(a) <= kStreamQueries ? Kind::Stream : Kind::Tree;
}

// The most tokens that a group walks: all of them, or what a window leaves (of any run of rows that a group has).
int64_t most_tokens(const AttendArgs& a, const Plan& pl) {
    const int64_t all = (int64_t)a.n * a.B;
    if (!a.window) return all;
    const int64_t rows = pl.chunk ? pl.rows / (a.Hq / a.Hk) + 2 : a.M, tile = pl.chunk ? 64 : 32;
    const int64_t some = (int64_t)a.sinks + a.window + rows + 2 * tile;      // (from and to a tile's edge)
    return some < all ? some : all;
}

// Items of a call, and so its workgroups, at most.
int64_t most_items(const AttendArgs& a, const Plan& pl) {
    return (int64_t)pl.slots * pl.rounds + (int64_t)a.S * a.Hk * pl.groups;
}

Plan plan_of(const AttendArgs& a, Kind kind) {
    const bool tree = kind != Kind::Stream;
    const int queries = queries_of(a);
    Plan pl;
    pl.chunk = kind == Kind::Chunk;
    pl.rows = tree ? 128 : 16;
    pl.groups = (queries + pl.rows - 1) / pl.rows;
    if (pl.rows > queries) pl.rows = queries;       // of one group
    // whole tiles (four waves take one each in the stream kernel), or whole blocks where a block's sum spans tiles
    pl.unit = tree ? 64 : 128;
    if (a.block_lse && a.B > 32) pl.unit = tree ? (a.B % 64 == 0 ? a.B : 2 * a.B) : 4 * a.B;
    // Two workgroups a CU, what the registers of the bf16 variants for 128 values a head leave room for (the stream
    // kernel's for 64 values would fit four, its e4m3 one for 128 three, which the plan does not use).  Items of a batch
    // are of uneven length where a run ends early, so more rounds than one even them out (64 sequences, FP8: 503 us
    // with 2, 463 with 4, 449 with 6), but a run has to be worth its start and its partial results (8 sequences of 5k
    // tokens, 13 rows: 75 us with 1, 91 with 2, 109 with 4).
    pl.slots = 2 * a.n_cu;
    pl.run = tree ? 2048 : 2560;
    const double most = (double)a.S * most_tokens(a, pl) * pl.groups * a.Hk / pl.slots / pl.run;
    pl.rounds = most < 1 ? 1 : (most < kRounds ? (int)most : kRounds);
    // (16 trees of 16 rows over up to 16416 tokens in 4 bits, where two tries leave 560 items for 512 places: 210 us, with
    // six 166.  bf16 and e4m3 caches without a window keep two, and with it the runs that they had.)
    pl.tries = a.cache.fp4 || a.window ? 6 : 2;
    pl.whole_from = 0;
    if (pl.chunk) {
        pl.rounds = 1;
        // Walks stay whole where they are up to 8192 tokens, so that one of a few groups is not much longer than the others,
        // and all groups fill half of the chip's places, or, of one sequence, are alike and the live ones fill three
        // quarters: the join and its sums cost more than the empty places.  In us, split and whole: one sequence of 32 heads
        // with 1100 rows (280 groups of 512 places), window 1024 71 and 63, 4096 163 and 155, none and a context of 32768
        // 916 and 1030; 1600 rows (400) 84 and 58, 180 and 157, 1088 and 1030; 4096 tokens of three sequences with up to 400
        // rows (300) 64 and 49, 3 x 4100 rows with a window of 1024 264 and 211.
        // How many are live is known on the device only.  Above 8192 tokens that decides, at the price of a join that may
        // find nothing to do: 16 live rows of n_rows 2048 over 131072 tokens took 3281 us where n_rows decided, 138 so.
        // Up to 8192 n_rows does (16 rows alone and of 2048: 27 and 99 us with a window of 4096), so that whole prompts need
        // neither join nor workspace.
        const int64_t items = (int64_t)a.S * a.Hk * pl.groups;
        if (most_tokens(a, pl) > 8192) {
            if (a.S == 1 && 4 * items >= 3 * pl.slots) pl.whole_from = (3 * pl.slots + 3) / 4;
        } else if (2 * items >= pl.slots) {
            pl.unit = kWhole;
            pl.tries = 0;       // nothing is left to fit
        }
    }
    pl.shortest = pl.unit;
    // A window of up to three of the shortest runs stays in one: the join's launch costs more than its split saves.  A call
    // of 1, 8, 64 sequences with 150 / 256 / 310 tokens in sight, us split and whole: 4 heads of 64 11 to 13 and 9 to 11
    // throughout; 32 heads of 128 14.5 and 12.7 / 14.2 / 12.9, 14.8 and 13.1 / 15.2 / 14.3, 21 / 26 / 28 and 19 / 24 / 25; the
    // same in 4 bits 12.7 and 9.8 / 10.7 / 10.3, 13.0 and 10.3 / 11.6 / 11.4, 15 / 16 / 17 and 12 / 14 / 14.  With 500 tokens
    // the one run is no shorter (4 heads 11.2) or longer (32 heads 14.1 and 16.9).
    if (a.window && !pl.chunk && !tree && most_tokens(a, pl) <= 3 * pl.unit) pl.shortest = 3 * pl.unit;
    pl.parts = most_items(a, pl);
    if (pl.whole_from > 0 && (int64_t)pl.slots * pl.rounds + pl.whole_from < pl.parts)      // (more live items have none)
        pl.parts = (int64_t)pl.slots * pl.rounds + pl.whole_from;
    return pl;
}

// Whether a sequence can have more than one run, so that there are partial results.
bool may_split(const AttendArgs& a, const Plan& pl) { return most_tokens(a, pl) > pl.shortest; }

size_t plan_bytes(const AttendArgs& a, const Plan& pl) {
    return may_split(a, pl) ? (size_t)(share_bytes(a.S) + pl.parts * pl.rows * (a.D + 2) * (int64_t)sizeof(float)) : 0;
}

template <int D, Held HELD>
void launch_fast(const AttendArgs& a, Kind kind, const Plan& pl, uint32_t grid, hipStream_t stream) {
    const BlockSize bs = block_size(a.B);
    if (kind == Kind::Stream) {
        if constexpr (HELD != FP4 || D == 128) {
            if (a.window) attend_stream_kernel<D, HELD, true><<<grid, 256, 0, stream>>>(a, pl, bs);
            else attend_stream_kernel<D, HELD, false><<<grid, 256, 0, stream>>>(a, pl, bs);
        }
    } else if (kind == Kind::Chunk) {
        launch_chunk<D, HELD>(a, pl, bs, grid, stream);
    } else if (!a.block_lse) attend_tree_kernel<D, HELD, 0><<<grid, 256, 0, stream>>>(a, pl, bs);
    else if (a.B == 8) attend_tree_kernel<D, HELD, 4><<<grid, 256, 0, stream>>>(a, pl, bs);
    else if (a.B == 16) attend_tree_kernel<D, HELD, 2><<<grid, 256, 0, stream>>>(a, pl, bs);
    else attend_tree_kernel<D, HELD, 1><<<grid, 256, 0, stream>>>(a, pl, bs);
}

// A workgroup for a row where a sequence has runs enough for its four waves,
// else D / 4 lanes (131072 tokens of one sequence in 64 runs are 32 rows; a
// batch's 65536 rows have few runs).
template <int D>
void launch_join(const AttendArgs& a, const Plan& pl, uint32_t rows, hipStream_t stream) {
    constexpr uint32_t per = 256 / (D / 4);
    if ((int64_t)pl.slots * pl.rounds > 8ll * a.S * a.Hk * pl.groups) attend_join_kernel<D><<<rows, 256, 0, stream>>>(a, pl);
    else {
        // Where walks may turn out whole, places' worth of workgroups that take the rows in turns: nothing to do is then
        // soon done (12000 rows of 32 heads: 20 us with a workgroup for each 8 of them, 4 so, of a call of 1288).
        const uint32_t all = (rows + per - 1) / per, some = 8u * (uint32_t)pl.slots;
        attend_join_rows_kernel<D><<<pl.whole_from > 0 && some < all ? some : all, 256, 0, stream>>>(a, pl, rows);
    }
}

}  // namespace
}  // namespace attend

using namespace attend;

size_t attend_workspace_bytes(const AttendArgs& a) {
    if (a.D != 64 && a.D != 128) return 0;
    // of a call without block_lse, whose runs can be the shorter; the cache may be of any type and layout
    const Kind many = a.window ? Kind::Chunk : Kind::Tree;
    const size_t tree = plan_bytes(a, plan_of(a, many));
    const size_t stream = queries_of(a) > (a.window ? kWindowQueries : kStreamQueries) ? 0 : plan_bytes(a, plan_of(a, Kind::Stream));
    return tree > stream ? tree : stream;
}

const char* attend_kernel_name(const AttendArgs& a) {
    switch (kind_of(a)) {
        case Kind::Stream: return "attend_stream_kernel";
        case Kind::Tree: return "attend_tree_kernel";
        case Kind::Chunk: return "attend_chunk_kernel";
        default: return "attend_plain_kernel";
    }
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.S * a.M;
    if (rows > 0x7FFFFFFF / a.Hq) return hipErrorInvalidConfiguration;
    const uint32_t row_grid = (uint32_t)(rows * a.Hq);
    const Kind kind = kind_of(a);
    auto threads_fit = [](int64_t threads) { return threads <= 0xFFFFFFFFll; };     // of a launch
    if (kind == Kind::Plain) {
        if (!threads_fit(256ll * row_grid)) return hipErrorInvalidConfiguration;
        const Held held = held_of(a.cache);
        auto launch = [&](auto held) {
            if (a.window) attend_plain_kernel<decltype(held)::value, true><<<row_grid, 256, 0, stream>>>(a);
            else attend_plain_kernel<decltype(held)::value, false><<<row_grid, 256, 0, stream>>>(a);
        };
        if (held == FP4) launch(std::integral_constant<Held, FP4>());
        else if (held == FP8) launch(std::integral_constant<Held, FP8>());
        else launch(std::integral_constant<Held, BF16>());
        return hipGetLastError();
    }
    const Plan pl = plan_of(a, kind);
    const bool split = may_split(a, pl);
    AttendArgs b = a;
    if (!split) b.ws = nullptr;
    // an XCD's items are numbered from the whole's eighth, rounded up
    // (and the chunk kernel's dead groups take workgroups behind the last)
    const int64_t grid = (most_items(a, pl) + 7) / 8 * 8 + (pl.chunk ? 8 : 0);
    // the join's launch too, before anything is enqueued (its kernel of 256 threads a row is for few rows)
    if (!grid_fits(grid) || !threads_fit(256 * grid) || (split && !threads_fit((int64_t)row_grid * (a.D / 4) + 256)))
        return hipErrorInvalidConfiguration;
    auto launch = [&](auto held) {
        if (a.D == 64) launch_fast<64, decltype(held)::value>(b, kind, pl, (uint32_t)grid, stream);
        else launch_fast<128, decltype(held)::value>(b, kind, pl, (uint32_t)grid, stream);
    };
    const Held held = held_of(a.cache);
    if (held == FP4) launch(std::integral_constant<Held, FP4>());
    else if (held == FP8) launch(std::integral_constant<Held, FP8>());
    else launch(std::integral_constant<Held, BF16>());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !split) return e;
    if (a.D == 64) launch_join<64>(b, pl, row_grid, stream);
    else launch_join<128>(b, pl, row_grid, stream);
    return hipGetLastError();
}

}  // namespace pred
