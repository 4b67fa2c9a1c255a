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

// Neighbouring tokens of a 4-bit cache lie in one line, and so do their scales: an XCD (b % 8) takes consecutive
// workgroups, so that its L2 gathers them.  The grid is a multiple of 8.
__device__ inline uint32_t xcd_order(uint32_t b, uint32_t grid) { return b % 8 * (grid / 8) + b / 8; }

// Heads a wave has in flight at once for each of its places (2048 tokens of 48
// heads of 128, four of them side by side in a wave: 14.1 us with 6, 15.8 with 3,
// 16.5 with 4, 16.3 with 12).
constexpr int kNormHeads = 6;

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

// What a wave keeps in LDS: the cosines and sines of its token's pairs, each
// worked out by one lane (every lane its own: 20 us instead of 14 for 2048
// tokens of 32 + 8 + 8 heads, 110 instead of 78 for the gradient), and the
// values that two lanes of a head exchange.
constexpr int kPairs = 256;         // of a head of 512
struct WaveLds {
    float c[kPairs], s[kPairs];
    float row[512];                 // 64 lanes of 8
};

__device__ inline void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// By all 64 lanes.
__device__ inline void set_angles(const RopeArgs& a, int64_t pos, WaveLds& lds, int lane) {
    for (int p = lane; p < a.rot / 2; p += 64) {
        const CosSin cs = cos_sin(a, pos, p);
        lds.c[p] = cs.c;
        lds.s[p] = cs.s;
    }
    wave_sync();
}

__device__ inline void read8(const float* from, float* x) {
    const float4 lo = *reinterpret_cast<const float4*>(from), hi = *reinterpret_cast<const float4*>(from + 4);
    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
}

// The cosines and sines of a lane's 8 values: of pairs (2 i, 2 i + 1) if INTER,
// else of each value, with the sine's sign.
template <bool INTER>
struct Angles {
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];

    __device__ inline void get(const WaveLds& lds, int rot, int d0) {
        const int half = rot / 2;
        if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = d0 / 2 + j < half ? d0 / 2 + j : 0;
                c[j] = lds.c[p];
                s[j] = lds.s[p];
            }
        } else if (rot % 16 == 0) {     // a piece's pairs are a piece
            const int p = d0 >= rot ? 0 : (d0 < half ? d0 : d0 - half);
            read8(lds.c + p, c);
            read8(lds.s + p, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = d0 < half ? -s[j] : s[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = d0 + j, p = d >= rot ? 0 : (d < half ? d : d - half);
                c[j] = lds.c[p];
                s[j] = d < half ? -lds.s[p] : lds.s[p];
            }
        }
    }

    // x turned; `first` is the head's first lane.  Every lane of the head calls it.
    __device__ inline void turn(float* x, int rot, int d0, WaveLds& lds, int lane, int first) const {
        if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (d0 + 2 * j >= rot) continue;
                const float u = x[2 * j], w = x[2 * j + 1];
                x[2 * j] = u * c[j] - w * s[j];
                x[2 * j + 1] = u * s[j] + w * c[j];
            }
        } else {
            float4* const mine = reinterpret_cast<float4*>(lds.row + 8 * lane);
            mine[0] = make_float4(x[0], x[1], x[2], x[3]);
            mine[1] = make_float4(x[4], x[5], x[6], x[7]);
            wave_sync();
            const int half = rot / 2;
            float y[8];
            if (rot % 16 == 0) {        // and its partners
                read8(lds.row + 8 * first + (d0 >= rot ? d0 : (d0 < half ? d0 + half : d0 - half)), y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = d0 + j;
                    y[j] = lds.row[8 * first + (d >= rot ? d : (d < half ? d + half : d - half))];
                }
            }
            wave_sync();
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
__global__ __launch_bounds__(256) void norm_rotate_kernel(NormArgs n, int pieces_any, int chunks, int deep) {
    __shared__ __attribute__((aligned(16))) WaveLds all_lds[4];
    const RopeArgs& a = n.rows;
    const int pieces = PIECES ? PIECES : pieces_any;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)xcd_order(blockIdx.x, gridDim.x) * 4 + wave, t = unit / chunks;
    if (t >= a.n_tokens) return;
    const int at_once = 64 / pieces, piece = lane % pieces, first = lane - piece, d0 = 8 * piece;
    const int heads = a.Hq + 2 * a.Hk, h0 = (int)(unit % chunks) * at_once * deep + lane / pieces;
    WaveLds& lds = all_lds[wave];
    const bool place = lane / pieces < at_once;
    const int64_t cache_off = token_offset(a, t);

    u32x4_t in[kNormHeads];
#pragma unroll
    for (int i = 0; i < kNormHeads; ++i) {
        const int h = h0 + i * at_once;
        in[i] = u32x4_t{0, 0, 0, 0};
        if (i < deep && h < heads && place) in[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(head_in(a, t, h) + d0));
    }
    if (a.rot) set_angles(a, a.positions[t], lds, lane);
    if (!place) return;
    Angles<INTER> angles;
    if (a.rot) angles.get(lds, a.rot, d0);
    float qw[8], kw[8];
    if (n.q.on) load_weight(n.q, d0, qw);
    if (n.k.on) load_weight(n.k, d0, kw);

#pragma unroll
    for (int i = 0; i < kNormHeads; ++i) {
        const int h = h0 + i * at_once;
        if (i >= deep || h >= heads) continue;
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
        if (a.rot && (is_q || is_k)) angles.turn(x, a.rot, d0, lds, lane, first);
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

// The gradient.  A workgroup a CU, of kGradWaves waves; a wave walks (token,
// heads) units a fixed distance apart, a lane keeps the sums of g h of its 8
// places, and a workgroup's come together in LDS: `part` gets a row of D a
// workgroup, which a second launch adds in a fixed order, so equal inputs give
// equal bits.
constexpr int kGradWaves = 16;
constexpr int kGradHeads = 2;        // as kNormHeads (78 us with 4, 76 with 2 and with 1)

template <int PIECES, bool INTER>
__global__ __launch_bounds__(64 * kGradWaves) void norm_rotate_backward_kernel(NormGradArgs n, int pieces_any, int chunks) {
    __shared__ __attribute__((aligned(16))) WaveLds all_lds[kGradWaves];
    const RopeArgs& a = n.rows;
    const int pieces = PIECES ? PIECES : pieces_any;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int at_once = 64 / pieces, piece = lane % pieces, first = lane - piece, d0 = 8 * piece;
    WaveLds& lds = all_lds[wave];
    float acc[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    const bool place = lane / pieces < at_once;
    if (place) load_weight(n.norm, d0, w);
    const uint32_t units = (uint32_t)(a.n_tokens * chunks);
    for (uint32_t unit = blockIdx.x * kGradWaves + wave; unit < units; unit += gridDim.x * kGradWaves) {
        const int64_t t = unit / chunks;
        const int h0 = (int)(unit % chunks) * at_once * kGradHeads + lane / pieces;
        u32x4_t xs[kGradHeads], gs[kGradHeads];
#pragma unroll
        for (int i = 0; i < kGradHeads; ++i) {
            const int h = h0 + i * at_once;
            xs[i] = gs[i] = u32x4_t{0, 0, 0, 0};
            if (h >= a.Hq || !place) continue;
            xs[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.q + t * a.q_stride + (int64_t)h * a.D + d0));
            gs[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(n.dy + t * n.dy_stride + (int64_t)h * a.D + d0));
        }
        if (a.rot) set_angles(a, a.positions[t], lds, lane);
        Angles<INTER> angles;
        if (a.rot) angles.get(lds, a.rot, d0);
#pragma unroll
        for (int i = 0; i < kGradHeads; ++i) {
            const int h = h0 + i * at_once;
            if (h >= a.Hq || !place) continue;
            float x[8], g[8];
            unpack8(xs[i], x);
            unpack8(gs[i], g);
            if (a.rot) angles.turn(g, a.rot, d0, lds, lane, first);
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
    float4* const mine = reinterpret_cast<float4*>(lds.row + 8 * lane);
    __syncthreads();
    mine[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    mine[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += 64 * kGradWaves) {
        float sum = 0.f;
        for (int v = 0; v < kGradWaves; ++v)
            for (int i = 0; i < at_once; ++i) sum += all_lds[v].row[8 * (i * pieces) + d];
        n.part[(int64_t)blockIdx.x * a.D + d] = sum;
    }
}

// dweight [D]: 16 columns a workgroup, 64 threads a column.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* part, int parts, int D, float* dweight) {
    __shared__ float sums[64][17];
    const int d = blockIdx.x * 16 + threadIdx.x % 16, lane = threadIdx.x / 16;
    float sum = 0.f;
    if (d < D) {
#pragma unroll 4
        for (int i = lane; i < parts; i += 64) sum += part[(int64_t)i * D + d];
    }
    sums[lane][threadIdx.x % 16] = sum;
    __syncthreads();
    if (lane != 0 || d >= D) return;
    for (int i = 1; i < 64; ++i) sum += sums[i][threadIdx.x];
    dweight[d] = sum;
}

// A wave a token (or one of `parts` of a token), a lane 8 values of a head at a time, kLoads of them in flight.
constexpr int kLoads = 4;

__global__ __launch_bounds__(256) void load_kernel(LoadArgs a, int pieces, int parts) {
    const int64_t unit = (int64_t)xcd_order(blockIdx.x, gridDim.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = unit / parts;
    const int part = (int)(unit % parts);
    if (t >= a.n_tokens) return;
    const int lane = threadIdx.x & 63;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.N * a.B) {
        if (slot != -1 && lane == 0 && part == 0) atomicOr(a.err, DEVERR_SLOT);
        return;
    }
    const int64_t token = slot / a.B * a.cache.block_stride + slot % a.B * a.cache.token_stride;
    const int items = 2 * a.Hk * pieces;
    for (int x0 = 64 * part + lane; x0 < items; x0 += 64 * kLoads * parts) {
        u32x4_t w[kLoads];
        uint32_t scale[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int x = x0 + 64 * parts * i;
            if (x >= items) continue;
            const int y = x / pieces, h = y < a.Hk ? y : y - a.Hk;
            const void* const from = y < a.Hk ? a.cache.k : a.cache.v;
            const int64_t off = token + h * a.cache.head_stride + x % pieces * 8;
            if (a.cache.fp4) {
                w[i][0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(from) + off / 2);
                scale[i] = (y < a.Hk ? a.cache.k_scales : a.cache.v_scales)[off / 32];
            } else if (a.cache.fp8) {
                const uint2 both = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(from) + off);
                w[i][0] = both.x;
                w[i][1] = both.y;
            } else {
                w[i] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(from) + off);
            }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int x = x0 + 64 * parts * i;
            if (x >= items) continue;
            const int y = x / pieces, h = y < a.Hk ? y : y - a.Hk;
            if (a.cache.fp4) {
                const float f = __uint_as_float(scale[i] << 23);
                const uint32_t bits = w[i][0];
                w[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, f, 0));
                w[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, f, 1));
                w[i][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, f, 2));
                w[i][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(bits, f, 3));
            } else if (a.cache.fp8) {
                const float f = y < a.Hk ? a.cache.k_scale : a.cache.v_scale;
                auto pair = [&](uint32_t word, auto hi) {
                    const auto v = __builtin_amdgcn_cvt_pk_f32_fp8((int)word, decltype(hi)::value);
                    return pack2(v[0] * f, v[1] * f);
                };
                w[i] = u32x4_t{pair(w[i][0], std::false_type()), pair(w[i][0], std::true_type()),
                               pair(w[i][1], std::false_type()), pair(w[i][1], std::true_type())};
            }
            __builtin_nontemporal_store(w[i], reinterpret_cast<u32x4_t*>((y < a.Hk ? a.k_out : a.v_out) +
                                                                         (t * a.Hk + h) * a.D + x % pieces * 8));
        }
    }
}

// of a launch, which has at most 2^32 - 1 threads (and these grids are rounded up to 32 waves)
constexpr int64_t kMostWaves = (1ll << 26) - 32;

int heads_a_wave(int D, int at_once) { return 64 / (D / 8) * at_once; }

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
    const int heads = a.rows.Hq + 2 * a.rows.Hk, pieces = a.rows.D / 8;
    // kNormHeads heads for each place of a wave, which share its angles and have their loads in flight together, or one
    // where that would give no more waves than the chip has SIMDs: 48 heads of 128 of 64 tokens 4.9 us with one, 7.8 with
    // six; 512 tokens 8.5 and 8.3, 2048 24.7 and 12.5; 16 heads into 4 bits without a rotation, 64 tokens 3.9 and 5.2,
    // 1024 5.0 and 5.5, 4096 11.4 and 8.3
    auto chunks_of = [&](int deep) { return (heads + heads_a_wave(a.rows.D, deep) - 1) / heads_a_wave(a.rows.D, deep); };
    const int deep = a.rows.n_tokens * chunks_of(kNormHeads) <= 1024 ? 1 : kNormHeads, chunks = chunks_of(deep);
    if (a.rows.n_tokens > kMostWaves / chunks) return hipErrorInvalidConfiguration;
    const uint32_t grid = (uint32_t)((a.rows.n_tokens * chunks + 31) / 32 * 8);
    norm_variant(pieces, a.rows.interleaved || !a.rows.rot, [&](auto p, auto inter) {
        norm_rotate_kernel<decltype(p)::value, decltype(inter)::value><<<grid, 256, 0, stream>>>(a, pieces, chunks, deep);
    });
    return hipGetLastError();
}

// Workgroups of the gradient, each with a row of sums: one for each of 256 CUs
// (its waves fill a CU), a wave each unit below that.
int64_t norm_grad_parts(int64_t n_tokens, int n_heads, int D) {
    const int per = heads_a_wave(D, kGradHeads), chunks = (n_heads + per - 1) / per;
    const int64_t units = n_tokens > (1ll << 40) ? (1ll << 40) : n_tokens * chunks;
    const int64_t groups = (units + kGradWaves - 1) / kGradWaves;
    return groups < 256 ? groups : 256;
}

hipError_t launch_norm_rotate_backward(const NormGradArgs& a, hipStream_t stream) {
    const int heads = a.rows.Hq, per = heads_a_wave(a.rows.D, kGradHeads), chunks = (heads + per - 1) / per, pieces = a.rows.D / 8;
    if (a.rows.n_tokens > 0x7FFFFFFFll / (chunks > 0 ? chunks : 1)) return hipErrorInvalidConfiguration;
    const int64_t parts = norm_grad_parts(a.rows.n_tokens, heads, a.rows.D);
    if (parts > 0) {
        norm_variant(pieces, a.rows.interleaved || !a.rows.rot, [&](auto p, auto inter) {
            norm_rotate_backward_kernel<decltype(p)::value, decltype(inter)::value>
                <<<(uint32_t)parts, 64 * kGradWaves, 0, stream>>>(a, pieces, chunks);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dweight) return hipSuccess;
    norm_weight_kernel<<<(a.rows.D + 15) / 16, 1024, 0, stream>>>(a.part, (int)parts, a.rows.D, a.dweight);
    return hipGetLastError();
}

hipError_t launch_load(const LoadArgs& a, hipStream_t stream) {
    // a wave a token, or where these are few one for each 64 of its pieces: 16 heads of 128 in 4 bits, 64 tokens 3.3 us in
    // parts and 4.9 without, 1024 4.3 and 5.3, 2048 5.7 and 5.6, 4096 7.6 and 6.9
    const int pieces = a.D / 8, all = (2 * a.Hk * pieces + 63) / 64, parts = a.n_tokens < 2048 ? all : 1;
    if (a.n_tokens > kMostWaves / parts) return hipErrorInvalidConfiguration;
    const int64_t grid = (a.n_tokens * parts + 31) / 32 * 8;
    load_kernel<<<(uint32_t)grid, 256, 0, stream>>>(a, pieces, parts);
    return hipGetLastError();
}

}  // namespace pred
