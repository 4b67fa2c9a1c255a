// Attention with a sliding window and sinks for more queries than the stream
// kernel takes: prompt chunks, whole prompts, chains of drafted tokens.
#include "attend.h"
#include "common.h"
#include "kernels.h"

namespace pred {
namespace attend {
namespace {

__device__ inline int live_groups(const AttendArgs& a, const Plan& pl, int drafted) {
    return (int)(((int64_t)drafted * (a.Hq / a.Hk) + pl.rows - 1) / pl.rows);
}

// A sequence's work: the most that a group of it walks, and the groups that have
// a live row.
struct ChunkWork {
    static constexpr bool kChunk = true;
    const AttendArgs& a;
    const Plan& pl;
    __device__ inline void operator()(int s, int& len, int& groups) const {
        const int tokens = kv_len_of(a.kv_len, s, (int64_t)a.n * a.B);
        const int some = (a.sinks + 63) / 64 * 64 + a.window + pl.rows / (a.Hq / a.Hk) + 1 + 64;
        groups = live_groups(a, pl, draft_len_of(a, s, tokens));
        len = groups == 0 ? 0 : (some < tokens ? some : tokens);
    }
};

// What the rows of groups without a live row get, by the workgroups behind the
// last item.  (As items between the others they left the XCDs work of uneven
// length: three prompts of 4100, 2470 and 2370 rows of n_rows 4100, 304 us, 249 so.)
__device__ inline void dead_groups(const AttendArgs& a, const Plan& pl, int spare, int spares) {
    const int lane = threadIdx.x & 63, g = a.Hq / a.Hk;
    const int64_t R = (int64_t)a.M * g;
    int64_t before = 0;     // of the sequences so far, kv heads counted
    for (int s0 = 0; s0 < a.S; s0 += 64) {
        int live = pl.groups;
        if (s0 + lane < a.S)
            live = live_groups(a, pl, draft_len_of(a, s0 + lane, kv_len_of(a.kv_len, s0 + lane, (int64_t)a.n * a.B)));
        uint64_t some = __ballot(live < pl.groups);
        for (; some != 0; some &= some - 1) {
            const int at = __builtin_ctzll(some), s = s0 + at, first = __builtin_amdgcn_readlane(live, at);
            const int64_t dead = (int64_t)(pl.groups - first) * a.Hk;
            for (int64_t x = (spare + spares - before % spares) % spares; x < dead; x += spares) {
                const int kvh = (int)(x % a.Hk), group = first + (int)(x / a.Hk);
                for (int y = threadIdx.x; y < pl.rows * (a.D / 8); y += 256) {
                    const int64_t r = (int64_t)pl.rows * group + y / (a.D / 8);
                    if (r >= R) break;
                    const int64_t row = ((int64_t)s * a.M + r / g) * a.Hq + kvh * g + r % g;
                    *reinterpret_cast<u32x4_t*>(a.out + row * a.D + y % (a.D / 8) * 8) = u32x4_t{0, 0, 0, 0};
                    if (a.lse && y % (a.D / 8) == 0) a.lse[row] = -INFINITY;
                }
                if (group == 0 && kvh == 0 && threadIdx.x == 0) {       // the sequence has no item
                    const int len = kv_len_of(a.kv_len, s, (int64_t)a.n * a.B);
                    check_lengths(a, s, len, 0);
                    if (a.ws) shares_of(a)[s] = Share{len, 1, 1 << 30, 1, 0};
                }
            }
            before += dead;
        }
    }
}

// ---------------------------------------------------------------- chunk kernel
//
// The tree kernel's layout (attend.hip): a workgroup has 128 queries of a kv
// head, consecutive in (row, query head), and walks tiles of 64 tokens through a
// double-buffered stage in LDS, each of its four waves with 32 queries, or, where
// up to 64 are live, two waves with the same 32 and half of each tile each.  Lane
// (n = lane % 32, f = lane / 32) owns query n.
//
// A group walks only the tiles that some row of it sees (Span): the sinks' and
// from its first row's window on, up to its last row.  Tiles that every row of
// the group sees whole need no masks; in the others values that are not finite
// become 0 (the tree kernel's drafted tokens).  bf16 goes straight into LDS and
// is cleaned there; narrow types are converted in registers on the way.
//
// A step: the loads of the next tile's values and of the keys of the one after it
// are issued; this tile's exponentials, and beside them, for the matrix cores,
// the next tile's scores; then the product with this tile's values, each read
// from LDS a step ahead.  So a wave has work for the vector units and for the
// matrix cores at a time (2048 rows of 8 queries for each of 8 heads of 128 on a
// window of 4096 tokens: 458 us with scores and exponentials of the same tile,
// 400 so; 400 -> 380 with the order in which turned() writes 4-bit values, which
// leaves 23% of LDS's cycles to bank conflicts for 38%, -> 375 with values a step
// ahead).
//
// With more than kWindowQueries queries per kv head the weights enter the value
// product as one bf16 term, 2^-8 of a weight off at most (the stream and tree
// kernels' two terms are half as many matrix instructions again: the call above 415 us
// for 325 from bf16, three prompts 244 for 202): an output is 2^-8 of the weighted
// mean of the absolute values off at most.  Where the values
// are of either sign that is about what the output's own rounding to bf16 adds
// (error against 64 bits 0.0023 relative, 0.0017 with the rounding alone).  Fewer
// queries, which come here where the cache's layout is not the stream kernel's, have
// two terms as they have there, so that a call's precision goes by its queries (one
// token of 32 heads of 64 over 131072 in 4 bits: 61 us with one term, 68 with two).
//
// Bound: the instructions of two waves a SIMD (the registers' limit).  Measured,
// that call (275 GFLOP of pairs that are seen), one after another: 329 us from a
// 4-bit cache, 836 TFLOP/s, 339 from bf16, 337 from e4m3, up to 8% more where a
// profiler's pauses let the clock fall; a matrix product of the library's reaches
// 1217.  Three prompts, 4 queries for each of 8 heads, window 1024: 207 us with 4100,
// 2469 and 2365 rows, 280 with 4100, 4095 and 3907.
// Short walks pay about 14 us of an item's start and end (18 tiles: 651 TFLOP/s).
// Tried and not kept: instruction orders laid down by hand, products k by k through
// both halves, wave priorities (all slower), eight waves of 32 queries (2%), 64
// queries a wave with one wave a SIMD (530 us, spills).  The stage's part of the
// time is about a quarter (286 us where its loads were left out).
template <int D, Held HELD>
__global__ __launch_bounds__(256, 2) void attend_chunk_kernel(AttendArgs a, Plan pl, BlockSize bs) {
    using T = TreeLds<D>;
    constexpr int RB = (int)(HELD == FP4 ? D / 2 : (HELD == FP8 ? D : 2 * D));      // bytes of a cache row
    constexpr int CR = RB / 16;                 // 16-byte pieces of it
    constexpr int NR = (64 * CR + 255) / 256;   // pieces a thread stages, of keys and of values
    constexpr int STEP = 256 / CR;              // tokens from one of them to the next: a multiple of 16
    constexpr int SPREAD = 2 * D / RB;          // pieces of an LDS row that one becomes
    constexpr int KS = D / 16, DT = D / 32;
    __shared__ __attribute__((aligned(16))) char lds[4 * T::kTile];     // keys 0, keys 1, values 0, values 1
    __shared__ int any_odd;         // a value of a tile that is not seen whole is not finite

    Item it = item_of(a, pl, blockIdx.x, ChunkWork{a, pl});
    if (it.slot < 0) {
        if (it.spare >= 0) dead_groups(a, pl, it.spare, it.spares);
        return;
    }
    {   // the longest walks first
        const int other = it.share.groups - 1 - it.group;
        it.slot += other - it.group;
        it.group = other;
    }
    it.share.len = kv_len_of(a.kv_len, it.s, (int64_t)a.n * a.B);
    const int s = it.s, kvh = it.kvh, len = it.share.len, drafted = draft_len_of(a, s, len);
    if (kvh == 0 && it.group == 0 && it.split == 0 && threadIdx.x == 0) {
        check_lengths(a, s, len, drafted);
        if (a.ws) shares_of(a)[s] = it.share;
    }
    const Span span = chunk_span(a, pl, len, drafted, it.group);
    const int runs = chunk_runs(span, it.share.run);
    if (it.split >= runs) return;
    // places of the walk
    const int v0 = it.split * it.share.run, v1 = v0 + it.share.run < span.end ? v0 + it.share.run : span.end;
    const int end = span.real_end(v1), ctx = len - drafted;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, f = lane >> 5;
    const int g = a.Hq / a.Hk, R = a.M * g;
    const int64_t group_r0 = (int64_t)pl.rows * it.group;
    const bool pairs = (int64_t)drafted * g - group_r0 <= 64;
    const int in_group = (pairs ? wave / 2 : wave) * 32, r0 = (int)group_r0 + in_group, r = r0 + n, i = r / g;
    const bool live = r < R && in_group + n < pl.rows && i < drafted;
    const bool wave_live = r0 < R && in_group < pl.rows && r0 / g < drafted;       // rows of a wave die from the end
    const int64_t row = ((int64_t)s * a.M + i) * a.Hq + kvh * g + r % g;
    const int pos = ctx + i, first = pos - a.window + 1;
    // of all live rows of the group, and of the wave
    auto last_row = [&](int r_last) { return r_last / g < drafted ? r_last / g : drafted - 1; };
    const int group_pos = ctx + (int)group_r0 / g, group_first = ctx + last_row((int)group_r0 + pl.rows - 1) - a.window + 1;
    const int wave_pos = ctx + r0 / g, wave_last = ctx + last_row(r0 + 31), wave_first = wave_last - a.window + 1;
    // every token of the 64 (32) from t on is seen by all rows from position `pos` on whose last window begins at `first`
    auto whole = [&](int t, int tokens, int lowest_pos, int highest_first) {
        return t + tokens - 1 <= lowest_pos && (t >= highest_first || t + tokens <= a.sinks);
    };

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

    // Staging, as in the tree kernel; t is a tile's first token.
    auto entry_of = [&](int t) {
        const int tok = t + lane;
        if (tok >= end) return -1;
        const int b = bs.block(tok);
        return table ? table[b] : b;
    };
    auto offset_of = [&](int t, int slot, uint64_t& nowhere) -> int64_t {
        const int tok = t + lane;
        const bool none = tok >= end || slot < 0 || slot >= a.N;
        nowhere = __ballot(none);
        return none ? 0 : bytes_of<HELD>(slot * a.cache.block_stride + (int64_t)(tok - bs.block(tok) * bs.B) * a.cache.token_stride);
    };
    const int my_tok = threadIdx.x / CR, my_piece = threadIdx.x % CR;       // and tokens STEP further on
    const bool mine_in = STEP * NR <= 64 || my_tok < 64;     // (64 values in 4 bits: half of the threads have a piece)
    // Keys and values of different tiles are on their way at a time.  `off` is where lane x's token lies (token x of the
    // tile).
    u32x4_t ks[NR], vs[NR];
    uint32_t k_sc[NR], v_sc[NR];        // a piece's scale byte
    auto place_of = [&](int64_t off, int x) -> int64_t {
        const int from = my_tok + STEP * x;
        return (int64_t)__shfl((int)(off >> 32), from) << 32 | (uint32_t)__shfl((int)off, from);
    };
    auto load_keys = [&](int64_t off) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int64_t o = place_of(off, x) + 16 * my_piece;
            ks[x] = *reinterpret_cast<const u32x4_t*>(kp + o);
            if constexpr (HELD == FP4) k_sc[x] = a.cache.k_scales[(head_off + o) >> 4];
        }
    };
    auto load_values = [&](int64_t off) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int64_t o = place_of(off, x) + 16 * my_piece;
            vs[x] = *reinterpret_cast<const u32x4_t*>(vp + o);
            if constexpr (HELD == FP4) v_sc[x] = a.cache.v_scales[(head_off + o) >> 4];
        }
    };
    // a thread's pieces of a narrow type as bf16 into LDS, `to` its first one's place
    auto store_pieces = [&](char* tile, int to, const u32x4_t* w, const uint32_t* sc) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            constexpr int kStep = STEP * T::kRow;
            if constexpr (HELD == FP4) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<u32x4_t*>(tile + (to ^ (16 * y)) + x * kStep) = fp4x8_to_bf16(w[x][y], sc[x]);
            } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    u32x4_t z;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        z[2 * e] = fp8x2_to_bf16<false>(w[x][2 * y + e]);
                        z[2 * e + 1] = fp8x2_to_bf16<true>(w[x][2 * y + e]);
                    }
                    *reinterpret_cast<u32x4_t*>(tile + (to ^ (16 * y)) + x * kStep) = z;
                }
            }
        }
    };
    const int turn = HELD == FP4 ? my_tok & (SPREAD - 1) : 0;       // of a thread's values: see turned()
    const int k_to = T::key(my_tok, SPREAD * my_piece), v_to = T::value(my_tok, SPREAD * my_piece) ^ (16 * turn);
    char* const keys = lds;
    char* const values = lds + 2 * T::kTile;
    auto store_keys = [&](int buf) {
        if (mine_in) store_pieces(keys + buf * T::kTile, k_to, ks, k_sc);
    };
    // t: the tile's first token; a value that not every row sees must be a number (a masked weight is 0)
    auto store_values = [&](int buf, int t, uint64_t nowhere) {
        if (!mine_in) return;
        if (nowhere != 0 || !whole(t, 64, group_pos, group_first)) {
            bool odd = false;
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const bool none = (nowhere >> (my_tok + STEP * x)) & 1;
                if constexpr (HELD == FP4) {
                    const bool bad = v_sc[x] == 255u;
                    odd |= bad && !none;
                    if (none || bad) {
                        vs[x] = u32x4_t{0, 0, 0, 0};
                        v_sc[x] = 0;
                    }
                }
#pragma unroll
                for (int y = 0; y < 4 && HELD == FP8; ++y) {
                    const uint32_t w = none ? 0u : vs[x][y];
                    vs[x][y] = finite_only_fp8(w);
                    odd |= vs[x][y] != w;
                }
            }
            if (odd) any_odd = 1;
        }
        if constexpr (HELD == FP4) {
#pragma unroll
            for (int x = 0; x < NR; ++x) vs[x] = turned(vs[x], turn);
        }
        store_pieces(values + buf * T::kTile, v_to, vs, v_sc);
    };
    // a bf16 tile straight into LDS: a lane fetches the piece that belongs in its place
    const int k_piece = my_piece ^ (D == 128 ? my_tok & 15 : (my_tok >> 1) & 7);
    const int v_piece = my_piece ^ (D == 128 ? (my_tok & 3) * 4 : ((my_tok >> 1) & 1) * 4);
    auto direct_tile = [&](char* tile, const char* from, int piece, int64_t off) {
        int64_t at[NR];
#pragma unroll
        for (int x = 0; x < NR; ++x) at[x] = place_of(off, x);
#pragma unroll
        for (int x = 0; x < NR; ++x)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) uint32_t*)(from + at[x] + 16 * piece),
                (__attribute__((address_space(3))) uint32_t*)(tile + (wave * (64 / CR) + STEP * x) * T::kRow), 16, 0, 0);
    };
    // values of such a tile, where this thread's pieces have come in: as store_values
    auto clean_values = [&](int buf, int t, uint64_t nowhere) {
        if (nowhere == 0 && whole(t, 64, group_pos, group_first)) return;
        bool odd = false;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            u32x4_t* const at = reinterpret_cast<u32x4_t*>(values + buf * T::kTile + (wave * (64 / CR) + STEP * x) * T::kRow + 16 * lane);
            const bool none = (nowhere >> (my_tok + STEP * x)) & 1;
            const u32x4_t in = *at;
            u32x4_t w;
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = none ? 0u : finite_only(in[y]);
            const bool differs = (w[0] != in[0]) | (w[1] != in[1]) | (w[2] != in[2]) | (w[3] != in[3]);
            odd |= differs && !none;
            if (differs) *at = w;
        }
        if (odd) any_odd = 1;
    };
    const int l16 = lane & 15;
    const int k_from = T::key(n, f);
    const int v_from = T::value(4 * f + l16 / 4, 2 * ((lane >> 4) & 1) + l16 % 4 / 2) + 8 * (l16 % 2);

    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16_t{};
    float m = kLowest, l = 0.f;
    const float scale = log2_scale(a);

    if (threadIdx.x == 0) any_odd = 0;
    __syncthreads();
    // A tile's scores are worked out one tile ahead, beside the exponentials of this one: the matrix cores and the vector
    // units each have work of a wave then.  So keys are a tile ahead of values in the stage.
    // HALVES = 2: the whole of every tile; 1: half `mine` of it.  TERMS: of a weight
    auto walk = [&](auto halves_, const int mine, auto terms_) {
        constexpr int HALVES = decltype(halves_)::value, TERMS = decltype(terms_)::value;
        f32x16_t x[HALVES];
        auto scores = [&](int buf) {
            const char* const kt = keys + buf * T::kTile + (HALVES == 1 ? 32 * mine * T::kRow : 0);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                f32x16_t acc = f32x16_t{};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const bf16x8_t key = __builtin_bit_cast(
                        bf16x8_t, *reinterpret_cast<const u32x4_t*>(kt + (k_from ^ (32 * k)) + 32 * h * T::kRow));
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key, q[k], acc, 0, 0, 0);
                }
                x[h] = acc;
            }
        };
        // tiles 0 and 1 (which may not be there: then its places are all nowhere)
        uint64_t nowhere, nowhere_1, nowhere_2 = 0;
        const int slot_0 = entry_of(span.real(v0)), slot_1 = entry_of(span.real(v0 + 64));
        int slot = entry_of(span.real(v0 + 128));
        const int64_t off = offset_of(span.real(v0), slot_0, nowhere);
        int64_t off_1 = offset_of(span.real(v0 + 64), slot_1, nowhere_1);
        if constexpr (HELD == BF16) {
            direct_tile(keys, kp, k_piece, off);
            direct_tile(values, vp, v_piece, off);
            direct_tile(keys + T::kTile, kp, k_piece, off_1);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            clean_values(0, span.real(v0), nowhere);
        } else {
            load_keys(off);
            load_values(off);
            store_keys(0);
            load_keys(off_1);
            store_values(0, span.real(v0), nowhere);
            store_keys(1);
        }
        __syncthreads();
        if (wave_live) scores(0);
        __syncthreads();        // the third tile's keys take the place of the first's
        for (int v = v0, buf = 0; v < v1; v += 64, buf ^= 1) {
            const bool more = v + 64 < v1, more_2 = v + 128 < v1;
            const int t = span.real(v), next = span.real(v + 64), next_2 = span.real(v + 128);
            int64_t off_2 = 0;
            if (more) {
                if (HELD == BF16) direct_tile(values + (buf ^ 1) * T::kTile, vp, v_piece, off_1);
                else load_values(off_1);
            }
            if (more_2) {
                off_2 = offset_of(next_2, slot, nowhere_2);
                if (HELD == BF16) direct_tile(keys + buf * T::kTile, kp, k_piece, off_2);
                else load_keys(off_2);
                slot = entry_of(span.real(v + 192));
            }
            uint64_t wrong = nowhere;       // invalid entries: tokens past the run's end are none
            if (t + 64 > end) wrong &= (1ull << (end - t)) - 1;
            if (wrong) wrong &= __ballot(t + lane < a.sinks || t + lane > group_pos - a.window);     // of tokens that some row sees
            if (wrong && wave == 0 && lane == 0) atomicOr(a.err, DEVERR_TABLE);
            if (wave_live) {
                const int th = t + 32 * mine;
                if (nowhere != 0 || !whole(th, 32 * HALVES, wave_pos, wave_first)) {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const uint32_t dead = (uint32_t)(nowhere >> (32 * (h + mine)));
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const int in = y % 4 + 8 * (y / 4) + 4 * f, tok = th + 32 * h + in;
                            const bool sees = ((dead >> in) & 1) == 0 && tok <= pos && (tok >= first || tok < a.sinks);
                            x[h][y] = sees ? x[h][y] : -INFINITY;
                        }
                    }
                }
                float tile_top = kLowest;
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
#pragma unroll
                    for (int y = 0; y < 16; y += 2) tile_top = max3(tile_top, x[h][y], x[h][y + 1]);
                tile_top *= scale;
                if (__ballot(tile_top > m + 8.f)) {
                    const float m_new = fmaxf(m, max_over_f(tile_top));
                    const float alpha = exp2_of(m - m_new);
                    m = m_new;
                    l *= alpha;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= alpha;
                }
                u32x4_t w[HALVES][2], rest[HALVES][2];      // the weights as second operands, and their second terms
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    float part_l[2] = {0.f, 0.f};
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        x[h][y] = exp2_of(__builtin_fmaf(x[h][y], scale, -m));
                        part_l[y / 8] += x[h][y];
                    }
                    l += part_l[0] + part_l[1];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const uint32_t pair = bf16_pair(x[h][2 * y], x[h][2 * y + 1]);
                        w[h][y / 4][y % 4] = pair;
                        if constexpr (TERMS == 2)
                            rest[h][y / 4][y % 4] = bf16_pair(rest_of<false>(x[h][2 * y], pair), rest_of<true>(x[h][2 * y + 1], pair));
                    }
                }
                scores(buf ^ 1);        // of the next tile (of what lies there, if there is none)
                const char* const vt = values + buf * T::kTile + (HALVES == 1 ? 32 * mine * T::kRow : 0);
                // 16 tokens a step, two transpose reads for 8 tokens' values of one d, a step ahead of the products
                bf16x8_t val[2][DT];
                auto read_values = [&](int step) {
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        struct { i16x4_t p[2]; } both;
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            both.p[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (lds_i16x4_t*)(vt + (v_from ^ (64 * d)) + (16 * step + 8 * z) * T::kRow));
                        val[step & 1][d] = __builtin_bit_cast(bf16x8_t, both);
                    }
                };
                read_values(0);
#pragma unroll
                for (int step = 0; step < 2 * HALVES; ++step) {
                    if (step + 1 < 2 * HALVES) read_values(step + 1);
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            val[step & 1][d], __builtin_bit_cast(bf16x8_t, w[step / 2][step % 2]), o[d], 0, 0, 0);
                    if constexpr (TERMS == 2) {
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                val[step & 1][d], __builtin_bit_cast(bf16x8_t, rest[step / 2][step % 2]), o[d], 0, 0, 0);
                    }
                }
            }
            if (HELD == BF16) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // in LDS before the barrier
                if (more) clean_values(buf ^ 1, next, nowhere_1);
            } else {
                if (more) store_values(buf ^ 1, next, nowhere_1);
                if (more_2) store_keys(buf);
            }
            nowhere = nowhere_1;
            nowhere_1 = nowhere_2;
            off_1 = off_2;
            __syncthreads();
        }
    };
    if (v0 < v1) {
        constexpr std::integral_constant<int, 1> one{};
        constexpr std::integral_constant<int, 2> two{};
        if (!pairs) walk(two, 0, one);
        else if (R > kWindowQueries) walk(one, wave % 2, one);
        else walk(one, wave % 2, two);
    }

    l = sum_over_f(l);
    bool lost = false;
    if constexpr (HELD == BF16) {
        float x = 0.f;      // NaN where a sum is not finite
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < 16; ++y) x = __builtin_fmaf(o[d][y], 0.f, x);
        lost = x != 0.f && l == l;
    }
    if (__ballot(lost) != 0 || any_odd) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            float sum[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) sum[y] = 0.f;
            for (int v = v0; v < v1; ++v) {
                if (pairs && (v - v0) / 32 % 2 != wave % 2) continue;       // the other wave's half
                const int tok = span.real(v);
                const char* const from = value_row<HELD>(a, bs, s, kvh, tok);
                if (from && tok <= pos && (tok >= first || tok < a.sinks)) {
#pragma unroll
                    for (int y = 0; y < 16; y += 4) add_not_finite<HELD>(sum + y, from, 32 * d + 2 * y + 4 * f);
                }
            }
#pragma unroll
            for (int y = 0; y < 16; ++y) o[d][y] = sum[y] == 0.f ? o[d][y] : sum[y];
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
                for (int y = 0; y < 16; ++y) x[(2 + 16 * d + y) * 64 + lane] = o[d][y];
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
            for (int y = 0; y < 16; ++y) o[d][y] = joined(o[d][y], mine, x[(2 + 16 * d + y) * 64 + lane], other);
    }
    if (pairs && runs == 1) {       // rows that no wave of the pairs has: past the last live one
        const int from = (int)group_r0 + 64, to = (int)group_r0 + pl.rows < R ? (int)group_r0 + pl.rows : R;
        for (int x = (wave / 2) * 64 + lane; x < (to - from) * (D / 8); x += 128) {
            const int y = from + x / (D / 8), d = x % (D / 8) * 8;
            const int64_t at = ((int64_t)s * a.M + y / g) * a.Hq + kvh * g + y % g;
            *reinterpret_cast<u32x4_t*>(a.out + at * D + d) = u32x4_t{0, 0, 0, 0};
            if (a.lse && d == 0) a.lse[at] = -INFINITY;
        }
    }
    if (r >= R || in_group + n >= pl.rows) return;
    const bool none = !live || l == 0.f;
    if (runs == 1) {
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

}  // namespace

template <int D, Held HELD>
void launch_chunk(const AttendArgs& a, const Plan& pl, const BlockSize& bs, uint32_t grid, hipStream_t stream) {
    attend_chunk_kernel<D, HELD><<<grid, 256, 0, stream>>>(a, pl, bs);
}
template void launch_chunk<64, BF16>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);
template void launch_chunk<64, FP8>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);
template void launch_chunk<64, FP4>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);
template void launch_chunk<128, BF16>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);
template void launch_chunk<128, FP8>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);
template void launch_chunk<128, FP4>(const AttendArgs&, const Plan&, const BlockSize&, uint32_t, hipStream_t);

}  // namespace attend
}  // namespace pred
