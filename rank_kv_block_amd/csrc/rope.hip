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
#include "rope.h"

namespace pred {
namespace {

// heads a lane turns with one set of cosines and sines (the e4m3 chunk: 13.8 us with 2, 12.6 with 3, 13.8 with 4, 13.2
// with 6)
constexpr int kHeads = 3;

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
