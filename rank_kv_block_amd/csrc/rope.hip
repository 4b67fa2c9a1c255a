// Rotary positions, and the store of a step's new keys and values into the
// paged cache.
//
//   out_a = m (x_a cos t - x_b sin t),  out_b = m (x_a sin t + x_b cos t),  t = position * f
//
// Angles.  f / (2 pi) is a 64-bit binary fraction of a turn, so position *
// turns modulo 2^64 is the angle modulo a turn, exactly: one integer product
// reduces any position, where a float32 product would lose the low bits of far
// positions.  Its top 32 bits become a float32 in [-1/2, 1/2) turns and go
// through sincospi.
//
// Bound: every value is read once and written once, 3 flops each, so a long
// call is HBM bound and a decode step's is one launch's latency.  A wave takes
// one token: a lane holds one 16-byte piece of a head (or, where pairs are half
// a rotation apart, the two pieces that turn together), the wave's lanes cover
// whole heads side by side, and a lane's cosines and sines serve the same
// pieces of up to kHeads heads, whose loads are all in flight at once.
//
// Measured: 8190 tokens of 64 heads of 128 (268 MB) 48 us, 5.6 TB/s, where a
// nontemporal copy of as much takes 42 us, 6.4 TB/s (52 us without the nontemporal
// loads and stores); 2048 tokens of 32 + 8 + 8 heads into an e4m3 cache (46 MB)
// 12.3 us; one token of 4 + 1 + 1 heads of 64 3.4 us.
#include "common.h"
#include "kernels.h"

namespace pred {
namespace {

// heads a lane turns with one set of cosines and sines (the e4m3 chunk: 13.8 us with 2, 12.6 with 3, 13.8 with 4, 13.2
// with 6)
constexpr int kHeads = 3;

struct CosSin {
    float c, s;
};

__device__ inline CosSin cos_sin(const RopeArgs& a, int64_t pos, int pair) {
    const uint64_t turn = (uint64_t)pos * a.turns[pair];
    const float half_turns = (float)(int32_t)(turn >> 32) * 0x1p-31f;
    CosSin r;
    float sn;
    sincospif(half_turns, &sn, &r.c);
    r.c *= a.mscale;
    r.s = a.backward ? -a.mscale * sn : a.mscale * sn;
    return r;
}

// float32 -> bf16, nearest even, one rounding.
__device__ inline uint32_t pack2(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

__device__ inline void unpack8(u32x4_t w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// value / scale clamped to e4m3's range (the conversion itself turns what is
// beyond it into NaN); NaN passes.
__device__ inline float to_fp8_range(float x, float scale) {
    x = x / scale;
    return x > 448.f ? 448.f : (x < -448.f ? -448.f : x);
}

// Eight values to d0 .. d0 + 7 of a cache row, or of a bf16 output row.
__device__ inline void store8(const float* x, void* row, int d0, bool fp8, float scale) {
    if (fp8) {
        int w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_fp8_range(x[4 * i], scale), to_fp8_range(x[4 * i + 1], scale),
                                                   0, false);
            w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_fp8_range(x[4 * i + 2], scale),
                                                   to_fp8_range(x[4 * i + 3], scale), w[i], true);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(row) + d0) = make_uint2(w[0], w[1]);
    } else {
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(row) + d0));
    }
}

// Where a token's cache rows begin (element offset), or -1 for one that stores
// nothing.
__device__ inline int64_t token_offset(const RopeArgs& a, int64_t t) {
    if (!a.Hk) return -1;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.N * a.B) {
        if (slot != -1) atomicOr(a.err, DEVERR_SLOT);
        return -1;
    }
    return slot / a.B * a.cache.block_stride + slot % a.B * a.cache.token_stride;
}

// Heads are numbered queries, keys, values.  The row a head reads, and the one
// it writes (null: nothing).
struct Rows {
    const uint16_t* in;
    void* out;
    bool turn, fp8;
    float scale;
};
__device__ inline Rows rows_of(const RopeArgs& a, int64_t t, int64_t cache_off, int h) {
    Rows r;
    const int64_t item = a.cache.fp8 ? 1 : 2;
    if (h < a.Hq) {
        r.in = a.q + t * a.q_stride + (int64_t)h * a.D;
        r.out = a.out + t * a.out_stride + (int64_t)h * a.D;
        r.turn = true;
        r.fp8 = false;
        r.scale = 1.f;
        return r;
    }
    r.fp8 = a.cache.fp8;
    const bool is_k = h < a.Hq + a.Hk;
    const int hk = h - a.Hq - (is_k ? 0 : a.Hk);
    r.in = (is_k ? a.k + t * a.k_stride : a.v + t * a.v_stride) + (int64_t)hk * a.D;
    r.out = cache_off < 0 ? nullptr
                          : static_cast<char*>(is_k ? a.cache.k : a.cache.v) +
                                (cache_off + hk * a.cache.head_stride) * item;
    r.turn = is_k;
    r.scale = is_k ? a.cache.k_scale : a.cache.v_scale;
    return r;
}

// One wave: one token, up to kHeads * (64 / pieces) heads.
template <bool INTER>
__global__ __launch_bounds__(256) void rotate_kernel(RopeArgs a, int pieces, int chunks) {
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t t = wave / chunks;
    if (t >= a.n_tokens) return;
    const int heads_at_once = 64 / pieces, lane = threadIdx.x & 63;
    const int piece = lane % pieces, heads = a.Hq + 2 * a.Hk;
    const int h0 = (int)(wave % chunks) * heads_at_once * kHeads + lane / pieces;
    if (lane / pieces >= heads_at_once) return;
    const int64_t cache_off = token_offset(a, t);

    // pieces that turn: INTER 8 values = 4 pairs; else 8 pairs, 8 values from each half of the rotation
    const int n_turning = INTER ? a.rot / 8 : a.rot / 16;
    const bool turning = piece < n_turning;
    const int d0 = turning ? 8 * piece : a.rot + 8 * (piece - n_turning);
    const int d1 = !INTER && turning ? d0 + a.rot / 2 : d0;

    u32x4_t lo[kHeads], hi[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * heads_at_once;
        if (h < heads) {
            const Rows r = rows_of(a, t, cache_off, h);
            lo[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(r.in + d0));
            if (!INTER) hi[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(r.in + d1));
        }
    }
    constexpr int kPairs = INTER ? 4 : 8;
    CosSin cs[kPairs];
    if (turning && h0 < a.Hq + a.Hk) {
        const int64_t pos = a.positions[t];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) cs[j] = cos_sin(a, pos, kPairs * piece + j);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * heads_at_once;
        if (h >= heads) continue;
        const Rows r = rows_of(a, t, cache_off, h);
        if (!r.out) continue;
        float x[8], y[8];
        unpack8(lo[i], x);
        if (INTER) {
            if (r.turn && turning) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = x[2 * j], w = x[2 * j + 1];
                    x[2 * j] = u * cs[j % kPairs].c - w * cs[j % kPairs].s;
                    x[2 * j + 1] = u * cs[j % kPairs].s + w * cs[j % kPairs].c;
                }
            }
            store8(x, r.out, d0, r.fp8, r.scale);
        } else {
            if (turning) {
                unpack8(hi[i], y);
                if (r.turn) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float u = x[j], w = y[j];
                        x[j] = u * cs[j % kPairs].c - w * cs[j % kPairs].s;
                        y[j] = u * cs[j % kPairs].s + w * cs[j % kPairs].c;
                    }
                }
                store8(y, r.out, d1, r.fp8, r.scale);
            }
            store8(x, r.out, d0, r.fp8, r.scale);
        }
    }
}

__device__ inline void store1(float x, void* row, int d, bool fp8, float scale) {
    if (fp8)
        static_cast<uint8_t*>(row)[d] =
            (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(to_fp8_range(x, scale), 0.f, 0, false);
    else
        static_cast<uint16_t*>(row)[d] = (uint16_t)pack2(x, 0.f);
}

// Rotations whose pairs do not fill 16-byte pieces (rot_dim not a multiple of
// 16, or 8 where interleaved): a lane per pair, or per value that does not turn,
// 2 bytes a load.  8190 tokens of 64 heads of 80, 20 of them turning (168 MB): 166
// us; with all 80 turning, in 16-byte pieces, 46.
__global__ __launch_bounds__(256) void rotate_pairs_kernel(RopeArgs a) {
    const int half = a.rot / 2, units = half + (a.D - a.rot), heads = a.Hq + 2 * a.Hk;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int unit = (int)(item % units), h = (int)(item / units % heads);
    const int64_t t = item / units / heads;
    if (t >= a.n_tokens) return;
    const Rows r = rows_of(a, t, token_offset(a, t), h);
    if (!r.out) return;
    if (unit >= half) {
        const int d = a.rot + unit - half;
        store1(bf16_lo(r.in[d]), r.out, d, r.fp8, r.scale);
        return;
    }
    const int da = a.interleaved ? 2 * unit : unit, db = a.interleaved ? da + 1 : da + half;
    float u = bf16_lo(r.in[da]), w = bf16_lo(r.in[db]);
    if (r.turn) {
        const CosSin cs = cos_sin(a, a.positions[t], unit);
        const float x = u;
        u = x * cs.c - w * cs.s;
        w = x * cs.s + w * cs.c;
    }
    store1(u, r.out, da, r.fp8, r.scale);
    store1(w, r.out, db, r.fp8, r.scale);
}

}  // namespace

hipError_t launch_rotate(const RopeArgs& a, hipStream_t stream) {
    const int heads = a.Hq + 2 * a.Hk;
    if (a.interleaved ? a.rot % 8 != 0 : a.rot % 16 != 0) {
        const int64_t units = a.rot / 2 + (a.D - a.rot);
        int64_t per = units * heads;
        if (a.n_tokens > (0x7FFFFFFFll * 256 - 255) / per) return hipErrorInvalidConfiguration;
        rotate_pairs_kernel<<<(uint32_t)((a.n_tokens * per + 255) / 256), 256, 0, stream>>>(a);
        return hipGetLastError();
    }
    const int pieces = a.interleaved ? a.D / 8 : a.rot / 16 + (a.D - a.rot) / 8;
    const int at_once = 64 / pieces * kHeads;
    const int chunks = (heads + at_once - 1) / at_once;
    if (a.n_tokens > (0x7FFFFFFFll * 4 - 3) / chunks) return hipErrorInvalidConfiguration;
    const uint32_t grid = (uint32_t)((a.n_tokens * chunks + 3) / 4);
    if (a.interleaved) rotate_kernel<true><<<grid, 256, 0, stream>>>(a, pieces, chunks);
    else rotate_kernel<false><<<grid, 256, 0, stream>>>(a, pieces, chunks);
    return hipGetLastError();
}

}  // namespace pred
