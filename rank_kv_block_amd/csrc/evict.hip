// Accumulated attention weight of cache blocks, and eviction by it.
#include "common.h"
#include "kernels.h"

namespace pred {
namespace {

// ---------------------------------------------------------------- weight
//
//   mass_out[s, b] = decay * mass[s, b] + sum_{accepted i, h} exp(block_lse[s, b, i, h] - lse[s, i, h])
//
// Bound: the accepted rows of block_lse are read once (4 bytes and one exp per
// row, head and block): HBM, or a launch's latency for one sequence.  LANES
// lanes share a block, a lane taking 4 heads (16 bytes) at a time, so a wave
// reads 64 / LANES blocks' rows side by side; rejected rows are not read.
//
// Measured: 8192 blocks of one sequence, one row of 32 heads (1.1 MB) 3.3 us; 64
// sequences of 2048 blocks, 16 rows of which 1 to 16 count (51 MB, in pieces of
// 128 bytes between rows that do not count; the memory reads 57) 17.9 us, 2.8
// TB/s: a block's rows follow one another, and each loads lse again.  Four rows'
// loads in flight a lane took 19.4 us.
template <int VEC>
__global__ __launch_bounds__(256) void weight_kernel(WeightArgs a, int lanes, uint32_t groups) {
    const int s = blockIdx.x / groups;
    const int per_group = 256 / lanes;
    const int64_t b = (int64_t)(blockIdx.x % groups) * per_group + threadIdx.x / lanes;
    const int sub = threadIdx.x % lanes;
    const int len = kv_len_of(a.kv_len, s, a.n * a.B);
    if (b == 0 && sub == 0 && a.kv_len && a.kv_len[s] != len) atomicOr(a.err, DEVERR_LEN);
    const int64_t used = ((int64_t)len + a.B - 1) / a.B;
    float sum = 0.f;
    if (b < used) {
        uint64_t rows = a.accepted ? a.accepted[s] : ~0ull;
        if (a.M < 64) rows &= (1ull << a.M) - 1;
        const float* x = a.block_lse + ((int64_t)s * a.n + b) * a.M * a.Hq;
        const float* z = a.lse + (int64_t)s * a.M * a.Hq;
        while (rows) {
            const int i = __builtin_ctzll(rows);
            rows &= rows - 1;
            for (int h = sub * VEC; h < a.Hq; h += lanes * VEC) {
                float xv[VEC], zv[VEC];
                if constexpr (VEC == 4) {
                    *reinterpret_cast<float4*>(xv) = *reinterpret_cast<const float4*>(x + (int64_t)i * a.Hq + h);
                    *reinterpret_cast<float4*>(zv) = *reinterpret_cast<const float4*>(z + (int64_t)i * a.Hq + h);
                } else {
                    xv[0] = x[(int64_t)i * a.Hq + h];
                    zv[0] = z[(int64_t)i * a.Hq + h];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float e = expf(xv[j] - zv[j]);
                    sum += zv[j] == -INFINITY ? 0.f : e;
                }
            }
        }
    }
    for (int m = lanes >> 1; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
    if (sub == 0 && b < a.n) {
        const int64_t at = (int64_t)s * a.n + b;
        if (b < used) a.mass_out[at] = a.decay * a.mass[at] + sum;
        else if (a.mass_out != a.mass) a.mass_out[at] = a.mass[at];
    }
}

// ---------------------------------------------------------------- evict
//
// One workgroup of 16 waves per sequence.  Wave w owns a contiguous range of
// the row and takes it 64 entries at a time, so an entry's place among those of
// its kind is the count of the waves before, plus the wave's running count,
// plus its rank in a ballot.  Everything is read before the first write, which
// is what lets an output be its input.
//
// The key below which everything goes is found 8 bits a step, from a histogram
// in LDS of the digits of the keys that still match.  Rows up to 1024 E keep
// their keys in registers (a protected entry's above every key); longer ones (E
// = 0) are copied to the workspace and read from there.  Bound: latency, of a
// row of 8 bytes an entry on one CU: 6.5 us for 64 rows of 2048, 11 us for one of
// 8192, 32 us for one of 32768; through the workspace 122 us for one of 65536 and
// 258 us for one of 131072.  (Fixing the key bit by bit from counts took 0.5 us a step: 12.8 and 44
// us.)
constexpr int kWaves = 16;
constexpr uint32_t kNoKey = 0xFFFFFFFFu;    // above every order key

// Sum over a wave, in every lane.
__device__ inline int wave_sum(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true);       // neighbours
    x += __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true);       // pairs
    x += __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, true);      // mirrored in 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, true);      // mirrored in 16
    auto a = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    x = (int)(a[0] + a[1]);
    auto b = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
    return (int)(b[0] + b[1]);
}

// Sum over a wave up to and with each lane.
__device__ inline int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);     // one to the right, in rows of 16
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);     // a row's last to the next row
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);     // the half's last to the other half
    return x;
}

// Where the entries of a wave go, 64 after 64.
struct Places {
    uint32_t key;       // keys below it go, and the first `ties` equal to it
    int ties, kept, used;
    int gone, equal;    // of the entries so far

    // the place of entry b of this lane, ~place if it goes
    __device__ inline int next(int b, uint32_t k) {
        uint64_t eq = __ballot(k == key);
        const int room = ties - equal, here = __popcll(eq);
        equal += here;
        if (here > room) {      // the tie that is cut, once a row, and those after it
            if (room <= 0) eq = 0;
            else
                while (__popcll(eq) > room) eq &= ~(1ull << (63 - __builtin_clzll(eq)));
        }
        const uint64_t out = eq | __ballot(k < key);
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(out >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)out, gone));
        gone += __popcll(out);
        const bool mine = (out >> (threadIdx.x & 63)) & 1;
        return mine ? ~(kept + before) : (b >= used ? b : b - before);
    }
};

template <int E>
__global__ __launch_bounds__(1024) void evict_kernel(EvictArgs a) {
    // a step's each; copies for lanes that would queue on one digit's address (masses share their leading bits), on
    // banks of their own
    constexpr int kCopies = E == 2 ? 2 : 8, kHist = 256 + 8;
    __shared__ __attribute__((aligned(16))) int hist[4][kCopies][kHist];
    __shared__ int ranks[2][kWaves];
    const int s = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = (int64_t)s * a.n;
    const int n_row = (int)a.n;
    const int len = kv_len_of(a.kv_len, s, a.n * a.B);
    if (threadIdx.x == 0 && a.kv_len[s] != len) atomicOr(a.err, DEVERR_LEN);
    const int used = (int)(((int64_t)len + a.B - 1) / a.B);
    const int lo = a.first < used ? a.first : used;
    const int hi = used - a.last > lo ? used - a.last : lo;    // candidates [lo, hi)
    const int64_t over = used > a.budget ? used - a.budget : 0;
    const int gone = over < hi - lo ? (int)over : hi - lo;

    constexpr int kHeld = E > 0 ? E : 1;
    const int steps = E > 0 ? E : (n_row + 64 * kWaves - 1) / (64 * kWaves);
    const int w0 = wave * 64 * steps;
    uint32_t keys[kHeld];
    int32_t* const copy_t = static_cast<int32_t*>(a.ws) + (E > 0 ? 0 : row);
    float* const copy_m = static_cast<float*>(a.ws) + (E > 0 ? 0 : (int64_t)a.S * a.n + row);
    auto key_of = [&](int b, float m) { return b >= lo && b < hi ? order_key(m) : kNoKey; };
    auto copied_key = [&](int b) { return b < n_row ? key_of(b, copy_m[b]) : kNoKey; };

    for (int x = threadIdx.x; x < 4 * kCopies * kHist; x += 1024) (&hist[0][0][0])[x] = 0;
    if constexpr (E > 0) {
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int b = w0 + 64 * e + lane;
            keys[e] = key_of(b, b < n_row ? a.mass[row + b] : 0.f);
        }
    } else {
        for (int e = 0; e < steps; ++e) {
            const int b = w0 + 64 * e + lane;
            if (b < n_row) {
                copy_t[b] = a.tables[row + b];
                copy_m[b] = a.mass[row + b];
            }
        }
    }
    __syncthreads();

    // the largest key with fewer than `gone` candidates below it
    uint32_t key = 0;
    int below = 0;      // candidates below the bits fixed so far
    if (gone > 0) {
        for (int step = 0; step < 4; ++step) {
            const int shift = 24 - 8 * step;
            // protected entries are above every key in each digit or an earlier one: counted, they change no digit below
            auto count = [&](uint32_t k) {
                if (step == 0 || (k ^ key) >> (shift + 8) == 0) atomicAdd(&hist[step][lane % kCopies][k >> shift & 255], 1);
            };
            if constexpr (E > 0) {
#pragma unroll
                for (int e = 0; e < kHeld; ++e) count(keys[e]);
            } else {
                for (int e = 0; e < steps; ++e) count(copied_key(w0 + 64 * e + lane));
            }
            __syncthreads();
            // every wave finds the digit for itself, four a lane
            int4 c = make_int4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int4 x = *reinterpret_cast<const int4*>(&hist[step][i][4 * lane]);
                c = make_int4(c.x + x.x, c.y + x.y, c.z + x.z, c.w + x.w);
            }
            const int own = c.x + c.y + c.z + c.w, upto = below + wave_scan(own);
            const int at = __builtin_ctzll(__ballot(upto >= gone));     // some lane: no more go than there are candidates
            int sum = upto - own, digit = 4 * lane;
            const int three[3] = {c.x, c.y, c.z};
            bool on = true;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                on = on && sum + three[i] < gone;
                sum += on ? three[i] : 0;
                digit += on;
            }
            key |= (uint32_t)__builtin_amdgcn_readlane(digit, at) << shift;
            below = __builtin_amdgcn_readlane(sum, at);
        }
    }

    // places: kept entries in order, then the evicted ones
    int wave_below = 0, wave_equal = 0;
    if constexpr (E > 0) {
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            wave_below += keys[e] < key;
            wave_equal += keys[e] == key;
        }
    } else {
        for (int e = 0; e < steps; ++e) {
            const uint32_t k = copied_key(w0 + 64 * e + lane);
            wave_below += k < key;
            wave_equal += k == key;
        }
    }
    wave_below = wave_sum(wave_below);
    wave_equal = wave_sum(wave_equal);
    if (lane == 0) {
        ranks[0][wave] = wave_below;
        ranks[1][wave] = wave_equal;
    }
    __syncthreads();
    Places p{key, gone - below, used - gone, used, 0, 0};
    for (int w = 0; w < wave; ++w) {
        p.gone += ranks[0][w];
        p.equal += ranks[1][w];
    }
    p.gone += p.equal < p.ties ? p.equal : p.ties;
    if constexpr (E > 0) {
        // in place of the keys; then the tables and the masses, each read whole before its first write
#pragma unroll
        for (int e = 0; e < kHeld; ++e) keys[e] = (uint32_t)p.next(w0 + 64 * e + lane, keys[e]);
        int32_t table[kHeld];
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int b = w0 + 64 * e + lane;
            table[e] = b < n_row ? a.tables[row + b] : 0;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int to = (int)keys[e] < 0 ? ~(int)keys[e] : (int)keys[e];
            if (w0 + 64 * e + lane < n_row) a.tables_out[row + to] = table[e];
        }
        float mass[kHeld];
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int b = w0 + 64 * e + lane;
            mass[e] = b < n_row ? a.mass[row + b] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int to = (int)keys[e] < 0 ? ~(int)keys[e] : (int)keys[e];
            if (w0 + 64 * e + lane < n_row) a.mass_out[row + to] = (int)keys[e] < 0 ? 0.f : mass[e];
        }
    } else {
        for (int e = 0; e < steps; ++e) {
            const int b = w0 + 64 * e + lane;
            const int place = p.next(b, copied_key(b)), to = place < 0 ? ~place : place;
            if (b < n_row) {
                a.tables_out[row + to] = copy_t[b];
                a.mass_out[row + to] = place < 0 ? 0.f : copy_m[b];
            }
        }
    }
    if (threadIdx.x == 0) {
        a.kv_len_out[s] = len - gone * a.B;
        a.evicted[s] = gone;
    }
}

constexpr int64_t kMaxHeld = 32768;     // entries of a row held in registers

}  // namespace

hipError_t launch_weight(const WeightArgs& a, hipStream_t stream) {
    const bool vec = a.Hq % 4 == 0 && aligned_to(a.lse, 16) && aligned_to(a.block_lse, 16);
    int lanes = 1;
    while (lanes < 64 && lanes * (vec ? 4 : 1) < a.Hq) lanes *= 2;
    const int64_t groups = (a.n + 256 / lanes - 1) / (256 / lanes);
    if (!grid_fits(groups) || !grid_fits(groups * a.S)) return hipErrorInvalidConfiguration;
    const uint32_t grid = (uint32_t)(groups * a.S);
    if (vec) weight_kernel<4><<<grid, 256, 0, stream>>>(a, lanes, (uint32_t)groups);
    else weight_kernel<1><<<grid, 256, 0, stream>>>(a, lanes, (uint32_t)groups);
    return hipGetLastError();
}

size_t evict_workspace_bytes(int64_t n, int64_t S) {
    return n <= kMaxHeld || S < 1 ? 0 : (size_t)n * (size_t)S * 8;
}

hipError_t launch_evict(const EvictArgs& a, hipStream_t stream) {
    const uint32_t grid = (uint32_t)a.S;
    if (a.n <= 2048) evict_kernel<2><<<grid, 1024, 0, stream>>>(a);
    else if (a.n <= 8192) evict_kernel<8><<<grid, 1024, 0, stream>>>(a);
    else if (a.n <= kMaxHeld) evict_kernel<32><<<grid, 1024, 0, stream>>>(a);
    else evict_kernel<0><<<grid, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace pred
