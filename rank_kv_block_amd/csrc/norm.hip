// Norms of queries and keys for each head, with the rotation and the store in
// the same pass; their gradient; rows stored without either (caches of every
// type, 4 bits among them); and cached tokens read back.
//
//   y = R(position) (x r (offset + w)),  r = 1 / sqrt(mean(x^2) + eps)
//
// over the D values of one head, R the rotation of rope.hip.  The gradient, with
// g = R^T dy, h = x r and u = g (offset + w):
//   dx = r (u - h mean(u h)),   dw = sum over tokens and heads of g h.
//
// A 4-bit cache holds e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), 32 of a head's values sharing a power of two: the smallest that
// keeps the largest of them within 6.  Keys that were normed or
// turned are rounded to bf16 before, so a key is the same whether it was stored
// in the pass or afterwards.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "rope.h"

namespace pred {
namespace {

// Heads a wave has in flight at once for each of its places.
constexpr int kNormHeads = 4;

// A wave takes one token: a lane holds 8 consecutive values (a piece) of a head,
// D / 8 lanes a head, heads side by side.  Half a rotation apart is another
// lane's piece, so those pairs meet through the wave's own part of LDS.

// The sum of a value over a head's lanes, in every one of them.  PIECES: lanes
// of a head, where they are a power of two; 0: `pieces` of them.
template <int PIECES>
__device__ inline float sum_of_head(float v, int pieces, int first) {
    if constexpr (PIECES == 0) {
        float sum = 0.f;
        for (int i = 0; i < pieces; ++i) sum += __shfl(v, first + i);
        return sum;
    } else {
        v += lane_xor<1>(v);
        v += lane_xor<2>(v);
        v += lane_xor<7>(v);
        if constexpr (PIECES >= 16) v += lane_xor<15>(v);
        if constexpr (PIECES >= 32) v += __shfl_xor(v, 16);
        return v;
    }
}

// The cosines and sines of a lane's 8 values: of pairs (2 i, 2 i + 1) if INTER,
// else of each value, with the sine's sign.
template <bool INTER>
struct Angles {
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];

    __device__ inline void set(const RopeArgs& a, int64_t pos, int d0) {
        const int half = a.rot / 2;
#pragma unroll
        for (int j = 0; j < (INTER ? 4 : 8); ++j) {
            const int d = INTER ? d0 + 2 * j : d0 + j;
            c[j] = 1.f;
            s[j] = 0.f;
            if (d < a.rot) {
                const CosSin cs = cos_sin(a, pos, INTER ? d / 2 : (d < half ? d : d - half));
                c[j] = cs.c;
                s[j] = INTER || d >= half ? cs.s : -cs.s;
            }
        }
    }

    // x turned; `row`: a place for the wave's 64 x 8 values, `first` the head's first lane.  Every lane of the head
    // calls it.
    __device__ inline void turn(float* x, int rot, int d0, float* row, int lane, int first) const {
        if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (d0 + 2 * j >= rot) continue;
                const float u = x[2 * j], w = x[2 * j + 1];
                x[2 * j] = u * c[j] - w * s[j];
                x[2 * j + 1] = u * s[j] + w * c[j];
            }
        } else {
            float4* const mine = reinterpret_cast<float4*>(row + 8 * lane);
            mine[0] = make_float4(x[0], x[1], x[2], x[3]);
            mine[1] = make_float4(x[4], x[5], x[6], x[7]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int half = rot / 2;
            float y[8];
            if (rot % 16 == 0) {        // a piece's partners are a piece
                const int at = 8 * first + (d0 >= rot ? d0 : (d0 < half ? d0 + half : d0 - half));
                const float4 lo = *reinterpret_cast<const float4*>(row + at), hi = *reinterpret_cast<const float4*>(row + at + 4);
                y[0] = lo.x, y[1] = lo.y, y[2] = lo.z, y[3] = lo.w, y[4] = hi.x, y[5] = hi.y, y[6] = hi.z, y[7] = hi.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = d0 + j;
                    y[j] = row[8 * first + (d >= rot ? d : (d < half ? d + half : d - half))];
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (d0 + j < rot) x[j] = x[j] * c[j] + y[j] * s[j];
        }
    }
};

// offset + w, or 1 without a weight
__device__ inline void load_weight(const HeadNorm& n, int d0, float* w) {
    if (!n.weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
        return;
    }
    unpack8(*reinterpret_cast<const u32x4_t*>(n.weight + d0), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] += n.offset;
}

// The scale byte of 32 values whose largest magnitude has these bf16 bits: e +
// 127 for the smallest 2^e with 6 * 2^e not below it, at least 2 (so that every
// value read is a normal number) and at most 252 (so that none is infinite:
// what is above 6 * 2^125 is cut there); 255 where a value is not finite.
__device__ inline uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7F80u) return 255u;
    const int e = (int)(top >> 7) - 2 + ((top & 127u) > 64u ? 1 : 0);
    return (uint32_t)(e < 2 ? 2 : (e > 252 ? 252 : e));
}

// 8 values of a head into a 4-bit row; its four lanes of 32 values come together.
__device__ inline void store8_fp4(const float* x, uint8_t* row, uint8_t* scales, int d0) {
    uint32_t w[4], top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = pack2(x[2 * i], x[2 * i + 1]);
        const uint32_t lo = w[i] & 0x7FFFu, hi = w[i] >> 16 & 0x7FFFu;
        top = max(top, max(lo, hi));
    }
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));
    const uint32_t byte = scale_byte(top);
    const float scale = __uint_as_float(byte << 23);
    uint32_t bits = 0;
    bits = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(bits, bf16_lo(w[0]), bf16_hi(w[0]), scale, 0);
    bits = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(bits, bf16_lo(w[1]), bf16_hi(w[1]), scale, 1);
    bits = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(bits, bf16_lo(w[2]), bf16_hi(w[2]), scale, 2);
    bits = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(bits, bf16_lo(w[3]), bf16_hi(w[3]), scale, 3);
    *reinterpret_cast<uint32_t*>(row + d0 / 2) = byte == 255u ? 0u : bits;
    if (d0 % 32 == 0) scales[d0 / 32] = (uint8_t)byte;
}

// Where head h (queries, keys, values in this order) of token t is read.
__device__ inline const uint16_t* head_in(const RopeArgs& a, int64_t t, int h) {
    if (h < a.Hq) return a.q + t * a.q_stride + (int64_t)h * a.D;
    h -= a.Hq;
    if (h < a.Hk) return a.k + t * a.k_stride + (int64_t)h * a.D;
    return a.v + t * a.v_stride + (int64_t)(h - a.Hk) * a.D;
}

template <int PIECES, bool INTER>
__global__ __launch_bounds__(256) void norm_rotate_kernel(NormArgs n, int pieces_any, int chunks) {
    __shared__ __attribute__((aligned(16))) float exchange[INTER ? 1 : 4][INTER ? 1 : 512];
    const RopeArgs& a = n.rows;
    const int pieces = PIECES ? PIECES : pieces_any;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave, t = unit / chunks;
    if (t >= a.n_tokens) return;
    const int at_once = 64 / pieces, piece = lane % pieces, first = lane - piece, d0 = 8 * piece;
    const int heads = a.Hq + 2 * a.Hk, h0 = (int)(unit % chunks) * at_once * kNormHeads + lane / pieces;
    if (lane / pieces >= at_once) return;
    float* const row = exchange[INTER ? 0 : wave];
    const int64_t cache_off = token_offset(a, t);

    u32x4_t in[kNormHeads];
#pragma unroll
    for (int i = 0; i < kNormHeads; ++i) {
        const int h = h0 + i * at_once;
        in[i] = u32x4_t{0, 0, 0, 0};
        if (h < heads) in[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(head_in(a, t, h) + d0));
    }
    Angles<INTER> angles;
    if (a.rot && h0 < a.Hq + a.Hk) angles.set(a, a.positions[t], d0);
    float qw[8], kw[8];
    if (n.q.on) load_weight(n.q, d0, qw);
    if (n.k.on) load_weight(n.k, d0, kw);

#pragma unroll
    for (int i = 0; i < kNormHeads; ++i) {
        const int h = h0 + i * at_once;
        if (h >= heads) continue;
        const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
        float x[8];
        unpack8(in[i], x);
        if (n.q.on | n.k.on) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
            const float mean = sum_of_head<PIECES>(ss, pieces, first) / a.D;
            if (is_q && n.q.on) {
                const float r = rsqrtf(mean + n.q.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= r * qw[j];
            }
            if (is_k && n.k.on) {
                const float r = rsqrtf(mean + n.k.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= r * kw[j];
            }
        }
        if (a.rot && (is_q || is_k)) angles.turn(x, a.rot, d0, row, lane, first);
        if (is_q) {
            store8(x, a.out + t * a.out_stride + (int64_t)h * a.D, d0, false, 1.f);
        } else if (cache_off >= 0) {
            const int hk = h - a.Hq - (is_k ? 0 : a.Hk);
            const int64_t off = cache_off + hk * a.cache.head_stride;
            void* const to = is_k ? a.cache.k : a.cache.v;
            if (a.cache.fp4)
                store8_fp4(x, static_cast<uint8_t*>(to) + off / 2, (is_k ? a.cache.k_scales : a.cache.v_scales) + off / 32, d0);
            else
                store8(x, static_cast<char*>(to) + off * (a.cache.fp8 ? 1 : 2), d0, a.cache.fp8,
                       is_k ? a.cache.k_scale : a.cache.v_scale);
        }
    }
}

// The gradient.  A wave walks (token, head) units a fixed distance apart; a lane
// keeps the sums of g h of its 8 places, and a workgroup's come together in
// LDS: `part` gets a row of D a workgroup, which a second launch adds in a fixed
// order, so equal inputs give equal bits.
template <int PIECES, bool INTER>
__global__ __launch_bounds__(256) void norm_rotate_backward_kernel(NormGradArgs n, int pieces_any, int chunks) {
    __shared__ __attribute__((aligned(16))) float exchange[4][512];
    const RopeArgs& a = n.rows;
    const int pieces = PIECES ? PIECES : pieces_any;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int at_once = 64 / pieces, piece = lane % pieces, first = lane - piece, d0 = 8 * piece;
    float* const row = exchange[wave];
    float acc[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    const bool place = lane / pieces < at_once;
    if (place) load_weight(n.norm, d0, w);
    for (int64_t unit = (int64_t)blockIdx.x * 4 + wave; unit < a.n_tokens * chunks && place; unit += (int64_t)gridDim.x * 4) {
        const int64_t t = unit / chunks;
        const int h0 = (int)(unit % chunks) * at_once * kNormHeads + lane / pieces;
        u32x4_t xs[kNormHeads], gs[kNormHeads];
#pragma unroll
        for (int i = 0; i < kNormHeads; ++i) {
            const int h = h0 + i * at_once;
            xs[i] = gs[i] = u32x4_t{0, 0, 0, 0};
            if (h >= a.Hq) continue;
            xs[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.q + t * a.q_stride + (int64_t)h * a.D + d0));
            gs[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(n.dy + t * n.dy_stride + (int64_t)h * a.D + d0));
        }
        Angles<INTER> angles;
        if (a.rot) angles.set(a, a.positions[t], d0);
#pragma unroll
        for (int i = 0; i < kNormHeads; ++i) {
            const int h = h0 + i * at_once;
            if (h >= a.Hq) continue;
            float x[8], g[8];
            unpack8(xs[i], x);
            unpack8(gs[i], g);
            if (a.rot) angles.turn(g, a.rot, d0, row, lane, first);
            float ss = 0.f, ux = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss += x[j] * x[j];
                ux += g[j] * w[j] * x[j];
            }
            ss = sum_of_head<PIECES>(ss, pieces, first);
            ux = sum_of_head<PIECES>(ux, pieces, first);
            const float r = rsqrtf(ss / a.D + n.norm.eps);
            const float mean = r * ux / a.D;        // of u h
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h_ = x[j] * r;
                acc[j] += g[j] * h_;
                x[j] = r * (g[j] * w[j] - h_ * mean);
            }
            store8(x, a.out + t * a.out_stride + (int64_t)h * a.D, d0, false, 1.f);
        }
    }
    if (!n.dweight) return;
    float4* const mine = reinterpret_cast<float4*>(row + 8 * lane);
    __syncthreads();
    mine[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    mine[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += 256) {
        float sum = 0.f;
        for (int v = 0; v < 4; ++v)
            for (int i = 0; i < at_once; ++i) sum += exchange[v][8 * (i * pieces) + d];
        n.part[(int64_t)blockIdx.x * a.D + d] = sum;
    }
}

// dweight [D]: 16 columns a workgroup, 16 threads a column.
__global__ __launch_bounds__(256) void norm_weight_kernel(const float* part, int64_t parts, int D, float* dweight) {
    __shared__ float sums[16][17];
    const int d = blockIdx.x * 16 + threadIdx.x % 16, lane = threadIdx.x / 16;
    float sum = 0.f;
    if (d < D)
        for (int64_t i = lane; i < parts; i += 16) sum += part[i * D + d];
    sums[lane][threadIdx.x % 16] = sum;
    __syncthreads();
    if (lane != 0 || d >= D) return;
    for (int i = 1; i < 16; ++i) sum += sums[i][threadIdx.x];
    dweight[d] = sum;
}

// A lane 8 values of a cached token's head.
__global__ __launch_bounds__(256) void load_kernel(LoadArgs a, int pieces) {
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (int64_t)2 * a.Hk * pieces, t = item / per;
    if (t >= a.n_tokens) return;
    const int in = (int)(item % per), d0 = in % pieces * 8, h = in / pieces % a.Hk;
    const bool is_k = in < a.Hk * pieces;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.N * a.B) {
        if (slot != -1 && in == 0) atomicOr(a.err, DEVERR_SLOT);
        return;
    }
    const int64_t off = slot / a.B * a.cache.block_stride + slot % a.B * a.cache.token_stride + h * a.cache.head_stride + d0;
    const void* const from = is_k ? a.cache.k : a.cache.v;
    u32x4_t w;
    if (a.cache.fp4) {
        const int bits = *reinterpret_cast<const int*>(static_cast<const uint8_t*>(from) + off / 2);
        const float scale = __uint_as_float((uint32_t)(is_k ? a.cache.k_scales : a.cache.v_scales)[off / 32] << 23);
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, scale, 0));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, scale, 1));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, scale, 2));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, scale, 3));
    } else if (a.cache.fp8) {
        const uint2 bits = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(from) + off);
        const float scale = is_k ? a.cache.k_scale : a.cache.v_scale;
        auto pair = [&](uint32_t word, auto hi) {
            const auto v = __builtin_amdgcn_cvt_pk_f32_fp8((int)word, decltype(hi)::value);
            return pack2(v[0] * scale, v[1] * scale);
        };
        w[0] = pair(bits.x, std::false_type());
        w[1] = pair(bits.x, std::true_type());
        w[2] = pair(bits.y, std::false_type());
        w[3] = pair(bits.y, std::true_type());
    } else {
        w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(from) + off);
    }
    *reinterpret_cast<u32x4_t*>((is_k ? a.k_out : a.v_out) + (t * a.Hk + h) * a.D + d0) = w;
}

int heads_a_wave(int D) { return 64 / (D / 8) * kNormHeads; }

// fn(lanes of a head where one of the variants has them, pairs side by side or not)
template <typename F>
void norm_variant(int pieces, bool inter, F fn) {
    auto with = [&](auto p) {
        if (inter) fn(p, std::true_type());
        else fn(p, std::false_type());
    };
    if (pieces == 8) with(std::integral_constant<int, 8>());
    else if (pieces == 16) with(std::integral_constant<int, 16>());
    else if (pieces == 32) with(std::integral_constant<int, 32>());
    else with(std::integral_constant<int, 0>());
}

}  // namespace

hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t stream) {
    const int heads = a.rows.Hq + 2 * a.rows.Hk, per = heads_a_wave(a.rows.D), chunks = (heads + per - 1) / per;
    if (a.rows.n_tokens > (0x7FFFFFFFll * 4 - 3) / chunks) return hipErrorInvalidConfiguration;
    const uint32_t grid = (uint32_t)((a.rows.n_tokens * chunks + 3) / 4);
    const int pieces = a.rows.D / 8;
    norm_variant(pieces, a.rows.interleaved || !a.rows.rot, [&](auto p, auto inter) {
        norm_rotate_kernel<decltype(p)::value, decltype(inter)::value><<<grid, 256, 0, stream>>>(a, pieces, chunks);
    });
    return hipGetLastError();
}

// Workgroups of the gradient: up to 1024, four for each of 256 CUs, so that
// their rows of sums stay few; a wave each unit below that.
int64_t norm_grad_parts(int64_t n_tokens, int n_heads, int D) {
    const int per = heads_a_wave(D), chunks = (n_heads + per - 1) / per;
    const int64_t units = n_tokens > (1ll << 40) ? (1ll << 40) : n_tokens * chunks, groups = (units + 3) / 4;
    return groups < 1024 ? groups : 1024;
}

hipError_t launch_norm_rotate_backward(const NormGradArgs& a, hipStream_t stream) {
    const int heads = a.rows.Hq, per = heads_a_wave(a.rows.D), chunks = (heads + per - 1) / per, pieces = a.rows.D / 8;
    if (a.rows.n_tokens > (0x7FFFFFFFll * 4 - 3) / (chunks > 0 ? chunks : 1)) return hipErrorInvalidConfiguration;
    const int64_t parts = norm_grad_parts(a.rows.n_tokens, heads, a.rows.D);
    if (parts > 0) {
        norm_variant(pieces, a.rows.interleaved || !a.rows.rot, [&](auto p, auto inter) {
            norm_rotate_backward_kernel<decltype(p)::value, decltype(inter)::value>
                <<<(uint32_t)parts, 256, 0, stream>>>(a, pieces, chunks);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dweight) return hipSuccess;
    norm_weight_kernel<<<(a.rows.D + 15) / 16, 256, 0, stream>>>(a.part, parts, a.rows.D, a.dweight);
    return hipGetLastError();
}

hipError_t launch_load(const LoadArgs& a, hipStream_t stream) {
    const int64_t per = (int64_t)2 * a.Hk * (a.D / 8);
    if (a.n_tokens > (0x7FFFFFFFll * 256 - 255) / per) return hipErrorInvalidConfiguration;
    load_kernel<<<(uint32_t)((a.n_tokens * per + 255) / 256), 256, 0, stream>>>(a, a.D / 8);
    return hipGetLastError();
}

}  // namespace pred
