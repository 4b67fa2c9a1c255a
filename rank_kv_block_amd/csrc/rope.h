// What the kernels share that turn and store rows of heads (rope.hip, norm.hip):
// a position's angles, the rows a head reads and writes, and the rounding to the
// cache's type.
#pragma once

#include "common.h"
#include "kernels.h"

namespace pred {
namespace {

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

__device__ inline void store1(float x, void* row, int d, bool fp8, float scale) {
    if (fp8)
        static_cast<uint8_t*>(row)[d] =
            (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(to_fp8_range(x, scale), 0.f, 0, false);
    else
        static_cast<uint16_t*>(row)[d] = (uint16_t)pack2(x, 0.f);
}

}  // namespace
}  // namespace pred
