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
// the row and reads it 64 entries at a time, so an entry's place among those of
// its kind is the count of the waves before, plus the wave's running count,
// plus a ballot's prefix.  With E > 0 a lane keeps its E entries in registers
// (rows up to 1024 E) and every pass runs from them; E = 0 reads them again
// from a copy in the workspace.  Reading everything before the first write is
// what lets an output be its input.
//
// The e-th lowest key is found bit by bit: 32 counts of the keys below a
// candidate.  Bound: latency (the row is 8 bytes an entry; 32 dependent
// counts).
constexpr int kWaves = 16;

struct Shared {
    int count[2][kWaves];
    int less[kWaves], equal[kWaves];
};

__device__ inline int sum_of(const int* c) {
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t += c[w];
    return t;
}

template <int E>
__global__ __launch_bounds__(1024) void evict_kernel(EvictArgs a) {
    __shared__ Shared sh;
    const int s = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = (int64_t)s * a.n;
    const int n_row = (int)a.n;
    const int given = a.kv_len[s];
    const int len = kv_len_of(a.kv_len, s, a.n * a.B);
    if (threadIdx.x == 0 && given != len) atomicOr(a.err, DEVERR_LEN);
    const int used = (int)(((int64_t)len + a.B - 1) / a.B);
    const int lo = a.first < used ? a.first : used;
    const int hi = used - a.last > lo ? used - a.last : lo;    // candidates [lo, hi)
    const int64_t over = used > a.budget ? used - a.budget : 0;
    const int gone = over < hi - lo ? (int)over : hi - lo;

    const int per_wave = E > 0 ? 64 * E : (n_row + 64 * kWaves - 1) / (64 * kWaves) * 64;
    const int w0 = wave * per_wave;
    constexpr int kHeld = E > 0 ? E : 1;
    int32_t held_t[kHeld];
    float held_m[kHeld];
    const int steps = E > 0 ? E : per_wave / 64;
    int32_t* const copy_t = static_cast<int32_t*>(a.ws) + (E > 0 ? 0 : row);
    float* const copy_m = static_cast<float*>(a.ws) + (E > 0 ? 0 : (int64_t)a.S * a.n + row);

    if constexpr (E > 0) {
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            const int b = w0 + 64 * e + lane;
            if (b < n_row) {
                held_t[e] = a.tables[row + b];
                held_m[e] = a.mass[row + b];
            }
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
    auto mass_of = [&](int e, int b) { return E > 0 ? held_m[E > 0 ? e : 0] : copy_m[b]; };
    auto table_of = [&](int e, int b) { return E > 0 ? held_t[E > 0 ? e : 0] : copy_t[b]; };

    // the key below which everything goes, and how many equal to it go too
    uint32_t key = 0;
    int ties = 0;
    if (gone > 0) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = key | (1u << bit);
            int c = 0;
#pragma unroll
            for (int e = 0; e < (E > 0 ? E : steps); ++e) {
                const int b = w0 + 64 * e + lane;
                c += __popcll(__ballot(b >= lo && b < hi && order_key(mass_of(e, b)) < cand));
            }
            int* const slot = sh.count[bit & 1];
            if (lane == 0) slot[wave] = c;
            __syncthreads();
            if (sum_of(slot) < gone) key = cand;
        }
    }
    // places: kept entries in order, then the evicted ones
    int below = 0, equal = 0;
    if (gone > 0) {
#pragma unroll
        for (int e = 0; e < (E > 0 ? E : steps); ++e) {
            const int b = w0 + 64 * e + lane;
            const bool in = b >= lo && b < hi;
            const uint32_t k = in ? order_key(mass_of(e, b)) : 0u;
            below += __popcll(__ballot(in && k < key));
            equal += __popcll(__ballot(in && k == key));
        }
    }
    if (lane == 0) {
        sh.less[wave] = below;
        sh.equal[wave] = equal;
    }
    __syncthreads();        // also: every read of the inputs is done before the first write below
    ties = gone - sum_of(sh.less);
    int below_before = 0, equal_before = 0;
    for (int w = 0; w < wave; ++w) {
        below_before += sh.less[w];
        equal_before += sh.equal[w];
    }
    const uint64_t before = (1ull << lane) - 1;
    const int kept = used - gone;
#pragma unroll
    for (int e = 0; e < (E > 0 ? E : steps); ++e) {
        const int b = w0 + 64 * e + lane;
        const bool in = gone > 0 && b >= lo && b < hi;
        const float m = b < n_row ? mass_of(e, b) : 0.f;
        const uint32_t k = order_key(m);
        const uint64_t lt = __ballot(in && k < key), eq = __ballot(in && k == key);
        const int eq_at = equal_before + __popcll(eq & before);
        // evicted entries before this one: those below the key, and of those equal to it the first `ties`
        const int out_before = below_before + __popcll(lt & before) + (eq_at < ties ? eq_at : ties);
        const bool out = in && (k < key || (k == key && eq_at < ties));
        if (b < n_row) {
            const int to = b >= used ? b : (out ? kept + out_before : b - out_before);
            a.tables_out[row + to] = table_of(e, b);
            a.mass_out[row + to] = out ? 0.f : m;
        }
        below_before += __popcll(lt);
        equal_before += __popcll(eq);
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
