// What the attention kernels share (attend.hip, window.hip): the types a cache
// holds, how the work is split over workgroups and its partial results lie, and
// the reads and roundings of their tiles.
#pragma once

#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace pred {
namespace attend {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// Start of a running maximum: finite, so that exp2(-inf - max) is 0 and not NaN
// for a masked score before the first real one.
constexpr float kLowest = -3.402823466e38f;

// How a cache holds its values.
enum Held : int { BF16, FP8, FP4 };
// bytes of x values (or of a stride of x)
template <Held HELD>
__host__ __device__ inline int64_t bytes_of(int64_t x) {
    return HELD == FP4 ? x / 2 : (HELD == FP8 ? x : 2 * x);
}
inline Held held_of(const CacheView& c) { return c.fp4 ? FP4 : (c.fp8 ? FP8 : BF16); }

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

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, bf16x2_t));
}

// x less its bf16 value, half HI of `pair`: exact, as one dot product.  The
// factor -1 is kept in a register: as an operand (-1, 0) the compiler writes
// the inline constant -1.0, which the instruction takes for (0, -1).
template <bool HI>
__device__ inline float rest_of(float x, uint32_t pair) {
    uint32_t minus_one = HI ? 0xBF800000u : 0x0000BF80u;
    asm("" : "+s"(minus_one));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, pair), __builtin_bit_cast(bf16x2_t, minus_one), x,
                                           false);
}

__device__ inline uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

__device__ inline float fp8_value(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }

// Values that are not finite.  A softmax weight is positive, so an infinite
// value that a row sees makes that element of its output the infinity, and two
// of opposite signs or a NaN make it NaN.  Sums of products give that only while
// the weight is held: one that underflows, or a matrix product's second term
// (which may be 0 or negative), turns the infinity into NaN.  So where a sum
// ends up not finite it becomes the sum of the values that are not, without
// weights; and sums are joined by joined().

// 0 for a number, else itself
__device__ inline float not_finite(float x) { return fabsf(x) < INFINITY ? 0.f : x; }

// a fa + b fb for factors in [0, 1]: an infinity stays one whatever its factor
__device__ inline float joined(float a, float fa, float b, float fb) {
    const float x = a * fa + b * fb;
    return x != x ? a + b : x;
}

// ---------------------------------------------------------------- splitting the work
//
// A workgroup takes an item: one group of `rows` queries of one kv head over
// one run of a sequence's tokens.  The lengths are on the device, so every
// workgroup works the split out for itself from all of them: with w_s = tokens
// of sequence s times its groups that have a live row, a run is about the sum
// of w_s over the items wanted, so the items are alike however uneven the
// sequences are.  A sequence of one run gets its result written by its items;
// of one with more the items write unnormalised sums, maximum and total, and
// a second launch joins them.
// With a window the rows of a sequence see its first `sinks` tokens and, each, the
// `window` newest up to itself.  What some row of i0 .. i1 sees lies in [0, head)
// and from head + skip on, both multiples of `unit`; a walk goes over the `end`
// tokens without the gap.
struct Span {
    int head, skip, end;
    __device__ inline int real(int v) const { return v < head ? v : v + skip; }
    // the real token after the last of a run that ends before v
    __device__ inline int real_end(int v) const { return v > head ? v + skip : v; }
};
__device__ inline Span span_of(const AttendArgs& a, int len, int drafted, int i0, int i1, int unit) {
    if (i1 < i0) return Span{0, 0, 0};
    const int first = len - drafted + i0 - a.window + 1, upto = len - drafted + i1 + 1;
    const int lo = first < 0 ? 0 : first / unit * unit, head = (a.sinks + unit - 1) / unit * unit;
    return lo > head ? Span{head, lo - head, upto - (lo - head)} : Span{upto, 0, upto};
}

struct Plan {
    int slots;      // workgroups the chip holds at once
    int rounds;     // at most this many times as many items; the runs' rounding adds at most one per sequence, head and
                    // group
    int run;        // shorter runs than this are not worth a round more: an item's start and its partial results
    int unit;       // a run is a multiple of this many tokens
    int shortest;   // and at least this long, a multiple of unit too
    int tries;      // at fitting the items into one round
    int rows;       // queries of a group
    int groups;     // groups of a kv head's queries
    bool chunk;     // of the chunk kernel: a group has a span of its own
    int whole_from; // and this many live items (or more) have whole walks; 0: what the run says
    int64_t parts;  // items that may have partial results
};
constexpr int kWhole = 1 << 30;     // a run above any number of tokens

// One sequence's share: `first` items (counting one kv head) before its own.
struct Share {
    int len, groups, run, runs, first;
};

struct Item {
    int s, kvh, group, split;
    Share share;
    int slot;       // index of its partial results; -1: no item
    bool last;      // the last group: it also writes what the rows of dead groups get
    int spare, spares;      // a workgroup behind an XCD's last item: which of how many
};

__device__ inline int runs_of(int len, int run) { return len > run ? (len + run - 1) / run : 1; }

// The tokens a group of sequence s walks and its groups, by the lengths alone.
struct DraftWork {
    static constexpr bool kChunk = false;
    const AttendArgs& a;
    const Plan& pl;
    __device__ inline void operator()(int s, int& len, int& groups) const {
        len = kv_len_of(a.kv_len, s, (int64_t)a.n * a.B);
        groups = (draft_len_of(a, s, len) * (a.Hq / a.Hk) + pl.rows - 1) / pl.rows;
        groups = groups < 1 ? 1 : groups;
    }
};

// Workgroup b of the grid, worked out by every wave alike.  Item f = ((first_s +
// split * groups) * Hk ..): an XCD (b % 8) takes consecutive items, so the
// groups that read the same bytes, and the heads whose bytes lie side by side,
// meet in one L2.  In the chunk kernel, whose walks are of uneven length, kv heads
// come first, so that an XCD has its part of every sequence (four prompts of
// uneven length without a window: 513 us by sequence, 400 by head; two of 12000
// and 7228 tokens, split, 2440 and 1885).
template <typename Work>
__device__ inline Item item_of(const AttendArgs& a, const Plan& pl, uint32_t b, Work work_of) {
    const int lane = threadIdx.x & 63;
    auto read = [&](int s, int& len, int& groups) {
        len = 0;
        groups = 0;
        if (s < a.S) work_of(s, len, groups);
    };
    int len0, groups0;      // the first 64 sequences' stay in registers
    read(lane, len0, groups0);
    auto sequence = [&](int s0, int& len, int& groups) {
        if (s0 == 0) {
            len = len0;
            groups = groups0;
        } else {
            read(s0 + lane, len, groups);
        }
    };
    auto wanted_run = [&]() {
        int64_t total = 0;
        for (int s0 = 0; s0 < a.S; s0 += 64) {
            int len, groups;
            sequence(s0, len, groups);
            total += (int64_t)len * groups;
        }
        if (a.S > 1)
            for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o);
        // (lane 0 has a single sequence's) the same in every lane from here on, in scalar registers
        total = ((int64_t)__builtin_amdgcn_readfirstlane((int)(total >> 32)) << 32 |
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)total)) * a.Hk;
        const int64_t per_slot = total / pl.slots, rounds = per_slot / pl.run;
        const int64_t items = (int64_t)pl.slots * (rounds < 1 ? 1 : (rounds < pl.rounds ? rounds : pl.rounds));
        const int64_t wanted = ((total + items - 1) / items + pl.unit - 1) / pl.unit * pl.unit;
        return (int)(wanted < pl.shortest ? pl.shortest : (wanted < 0x7FFFFFFF ? wanted : 0x7FFFFFFF));
    };
    auto items_of = [&](int run) {
        int count = 0;      // of one kv head
        for (int s0 = 0; s0 < a.S; s0 += 64) {
            int len, groups;
            sequence(s0, len, groups);
            count += groups * runs_of(len, run);
        }
        if (a.S > 1)
            for (int o = 32; o >= 1; o >>= 1) count += __shfl_xor(count, o);
        return (uint32_t)__builtin_amdgcn_readfirstlane(count) * a.Hk;
    };
    const bool whole = Work::kChunk && (pl.tries == 0 || (pl.whole_from > 0 && items_of(kWhole) >= (uint32_t)pl.whole_from));
    int run = whole ? kWhole : wanted_run();
    uint32_t all = items_of(run);
    // Every sequence's last run is a part of one, so the items are a few more than wanted.  Where they pass one round
    // by up to a quarter, runs a little longer do without the second, nearly empty one (8 sequences of 5k tokens, 13
    // rows: 78 us without, 70 with; with more rounds there is nothing to gain).
    const uint32_t one = (uint32_t)pl.slots;
    int longer = run;
    for (uint32_t tries = 0, now = all; !whole && tries < (uint32_t)pl.tries && all > one && all - one <= one / 4; ++tries) {
        const int64_t fits = ((int64_t)longer * now / one + pl.unit) / pl.unit * pl.unit;
        longer = (int)(fits < 0x40000000 ? fits : 0x40000000 / pl.unit * pl.unit);
        now = items_of(longer);
        if (now <= one) {
            run = longer;
            all = now;
        }
    }
    const uint32_t each = (all + 7) / 8, f = b % 8 * each + b / 8;
    Item it{};
    it.slot = -1;
    it.spare = (int)(b - 8 * each);
    it.spares = (int)(gridDim.x - 8 * each);
    if (b / 8 >= each || f >= all) return it;
    const uint32_t of_head = all / a.Hk, at_f = Work::kChunk ? f % of_head : f / a.Hk;      // among one kv head's items
    int before = 0;
    for (int s0 = 0; s0 < a.S; s0 += 64) {
        int len, groups;
        sequence(s0, len, groups);
        const int own = groups * runs_of(len, run);
        int upto = own;
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(upto, o);
            if (lane >= o) upto += x;
        }
        const uint64_t past = __ballot((uint32_t)(before + upto) > at_f);
        if (past) {
            const int at = __builtin_ctzll(past);
            it.s = s0 + at;
            it.share.first = __builtin_amdgcn_readlane(before + upto - own, at);
            it.share.len = __builtin_amdgcn_readlane(len, at);
            it.share.groups = __builtin_amdgcn_readlane(groups, at);
            break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    it.share.runs = runs_of(it.share.len, run);
    // the sequence's runs, evened out
    const int even_run = (it.share.len + it.share.runs - 1) / it.share.runs;
    it.share.run = it.share.runs == 1 ? run : (even_run + pl.unit - 1) / pl.unit * pl.unit;
    const uint32_t before_it = (uint32_t)it.share.first * a.Hk;
    if constexpr (Work::kChunk) {
        const uint32_t in = at_f - (uint32_t)it.share.first;
        it.group = (int)(in % it.share.groups);
        it.split = (int)(in / it.share.groups);
        it.kvh = (int)(f / of_head);
        it.slot = (int)(before_it + (it.split * a.Hk + it.kvh) * it.share.groups + it.group);
    } else {
        uint32_t in = f - before_it;
        it.slot = (int)f;
        it.group = (int)(in % it.share.groups);
        in /= it.share.groups;
        it.kvh = (int)(in % a.Hk);
        it.split = (int)(in / a.Hk);
    }
    it.last = it.group == it.share.groups - 1;
    return it;
}

// Workspace: each sequence's share, then [parts, rows, D] sums, then [parts,
// rows] (maximum, total).
__device__ inline Share* shares_of(const AttendArgs& a) { return static_cast<Share*>(a.ws); }
__host__ __device__ inline int64_t share_bytes(int64_t S) { return (S * (int64_t)sizeof(Share) + 15) / 16 * 16; }
__device__ inline float* part_sums(const AttendArgs& a, const Plan& pl, int64_t slot) {
    return reinterpret_cast<float*>(static_cast<char*>(a.ws) + share_bytes(a.S)) + slot * pl.rows * a.D;
}
__device__ inline float2* part_stats(const AttendArgs& a, const Plan& pl, int64_t slot) {
    return reinterpret_cast<float2*>(part_sums(a, pl, pl.parts)) + slot * pl.rows;
}

// Turns a product q k into units of log2: above 0, so that a masked -inf stays
// one (the queries carry a negative scale's sign).  A scale of 0, which weighs
// every token alike, is 2^-120 here: products below 2^96 differ by less than
// 2^-24 then.
__device__ inline float log2_scale(const AttendArgs& a) {
    return fmaxf(fabsf(a.scale) * a.cache.k_scale * kLog2e, 0x1p-120f);
}

// x, or -x where scale is negative
__device__ inline bf16x8_t signed_by(float scale, bf16x8_t x) {
    const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;
    return __builtin_bit_cast(bf16x8_t, __builtin_bit_cast(u32x4_t, x) ^ (u32x4_t){flip, flip, flip, flip});
}

// two e4m3 values (bytes 0, 1 or 2, 3 of w) as two bf16, exact
template <bool HI>
__device__ inline uint32_t fp8x2_to_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI));
}

// eight e2m1 values as eight bf16 times the power of two of a scale byte, exact
__device__ inline u32x4_t fp4x8_to_bf16(uint32_t w, uint32_t scale_byte) {
    const float scale = __uint_as_float(scale_byte << 23);
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
}

// Division of a token's index by the block size: one 64-bit product.  With
// 2^(s-1) < B <= 2^s and magic = ceil(2^(31+s) / B), magic * B - 2^(31+s) < B <=
// 2^s, so t * magic >> (31 + s) is t / B for every t < 2^31.
struct BlockSize {
    int B, shift;           // shift = 31 + s
    uint32_t magic;
    __host__ __device__ inline int block(int t) const { return (int)((uint64_t)(uint32_t)t * magic >> shift); }
};

inline BlockSize block_size(int B) {
    int s = 0;
    while (s < 31 && (1u << s) < (uint32_t)B) ++s;
    const uint64_t one = 1ull << (31 + s);
    return BlockSize{B, 31 + s, (uint32_t)((one + B - 1) / B)};
}

// The larger of three, one instruction where `a` is known to be a number.
__device__ inline float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// w with its halves that are not finite set to 0
__device__ inline uint32_t finite_only(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}

// the same for four e4m3 values, whose only such pattern is NaN (0x7F, 0xFF)
__device__ inline uint32_t finite_only_fp8(uint32_t w) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (((w >> i) & 0x7Fu) == 0x7Fu) w &= ~(0xFFu << i);
    return w;
}

// A masked weight is 0, and 0 times a value that is not finite would be NaN in
// the matrix cores.  So drafted tokens' values enter the products with 0 in the
// place of what is not finite.  A run that holds any, or whose sums are not
// finite (every row sees the whole context), walks its tokens once more and
// takes what is not finite from there.  (e4m3 and a 4-bit cache have no
// infinities, and a NaN of the context needs no walk.)

// Adds what is not finite among the 4 values from d on of a token's head, `row` from value_row.
template <Held HELD>
__device__ inline void add_not_finite(float* sum, const char* row, int d) {
    if constexpr (HELD == FP4) {
        if ((uint8_t)row[d / 32] == 255u)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = NAN;
    } else if constexpr (HELD == FP8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + d);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (((w >> (8 * e)) & 0x7Fu) == 0x7Fu) sum[e] = NAN;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 2 * d);
        sum[0] += not_finite(bf16_lo(w.x));
        sum[1] += not_finite(bf16_hi(w.x));
        sum[2] += not_finite(bf16_lo(w.y));
        sum[3] += not_finite(bf16_hi(w.y));
    }
}
// The values of a token's head (of a 4-bit cache their scales), null where its block has an invalid entry.
template <Held HELD>
__device__ inline const char* value_row(const AttendArgs& a, const BlockSize& bs, int s, int kvh, int tok) {
    const int b = bs.block(tok);
    const int64_t slot = a.tables ? a.tables[(int64_t)s * a.n + b] : b;
    if (slot < 0 || slot >= a.N) return nullptr;
    const int64_t at = slot * a.cache.block_stride + (int64_t)(tok - b * bs.B) * a.cache.token_stride +
                       (int64_t)kvh * a.cache.head_stride;
    if constexpr (HELD == FP4) return reinterpret_cast<const char*>(a.cache.v_scales) + at / 32;
    return static_cast<const char*>(a.cache.v) + bytes_of<HELD>(at);
}

// Queries per kv head that the stream kernel takes with a window: one group (16 queries over 16 sequences' windows of
// 4096: 58 us and 57 with the chunk kernel, from a 4-bit cache 30 and 48; of one sequence 17 and 20, of 64 187 and 206).
// Up to so many a weight has two bf16 terms in the chunk kernel too.
constexpr int kWindowQueries = 16;

// LDS tiles of the tree and chunk kernels.
template <int D>
struct TreeLds {
    static constexpr int kRow = 2 * D;              // bytes of a row
    static constexpr int kPieces = kRow / 16;
    static constexpr int kTile = 64 * kRow;
    // byte offset of 16-byte piece `piece` of row `row`
    __device__ static inline int key(int row, int piece) {
        return row * kRow + 16 * (piece ^ (D == 128 ? row & 15 : (row >> 1) & 7));
    }
    __device__ static inline int value(int row, int piece) {
        return row * kRow + 16 * (piece ^ (D == 128 ? (row & 3) * 4 : ((row >> 1) & 1) * 4));
    }
};

// A staged piece of a narrower type becomes 2 (e4m3) or 4 (4 bits) pieces side by side in an LDS row, written one a step:
// in step y the one at `to ^ (16 * y)`.  The permutation of the values' rows is of groups of four pieces, so in one order
// for all lanes a step's writes of a 4-bit cache would put 4 lanes of 16 on one bank.  So lanes of neighbouring rows take
// their values' pieces in orders of their own: the place is turned by the row's low bits (`to ^ (16 * turn)`), and the
// piece's words with it.  2048 rows on 32768 tokens in 4 bits: bank conflicts 38% of the cycles in which LDS is at work
// without, 23% so (what is left was not taken further), 333 us and 321.  From e4m3 22% either way, and 331 us without, 336
// turned; so it goes without.
__device__ inline u32x4_t turned(u32x4_t w, int turn) {
    if (turn & 1) w = u32x4_t{w[1], w[0], w[3], w[2]};
    if (turn & 2) w = u32x4_t{w[2], w[3], w[0], w[1]};
    return w;
}

// max / sum over the two lanes of a query
__device__ inline float max_over_f(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ inline float sum_over_f(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

// What group `group` of a sequence walks in the chunk kernel, and its runs.
__device__ inline Span chunk_span(const AttendArgs& a, const Plan& pl, int len, int drafted, int group) {
    const int g = a.Hq / a.Hk, last = (pl.rows * (group + 1) - 1) / g;
    return span_of(a, len, drafted, pl.rows * group / g, last < drafted ? last : drafted - 1, 64);
}
__device__ inline int chunk_runs(const Span& span, int run) { return runs_of(span.end, run); }

// The chunk kernel (window.hip).
template <int D, Held HELD>
void launch_chunk(const AttendArgs& a, const Plan& pl, const BlockSize& bs, uint32_t grid, hipStream_t stream);

}  // namespace attend
}  // namespace pred
