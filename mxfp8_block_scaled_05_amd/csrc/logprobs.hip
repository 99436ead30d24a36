// Log-probabilities of given tokens, entropy and the likeliest tokens of rows
// of logits, and the gradient of the first two.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;         // threads of the gradient's and of split rows' blocks
constexpr int kWide = 1024;         // threads of a block that has a long row to itself
constexpr int kUnroll = 4;          // 16-byte loads of a thread in flight
constexpr float kLowest = -3.402823466e38f;

// Statistics of a set of logits: m = max x, s = sum e^((x - m) / temp),
// w = sum e^(..) (x - m) c with c = log2(e) / temp (so w is in base 2).
// A set without a logit above -Inf has s = 0.
struct Stats {
    float m, s, w;
};

// joins two sets; both corrections carry the same sign, so nothing cancels
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b, float c) {
    Stats r;
    r.m = __builtin_fmaxf(a.m, b.m);
    const float da = __builtin_fmaxf((a.m - r.m) * c, -1000.0f), db = __builtin_fmaxf((b.m - r.m) * c, -1000.0f);
    const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
    r.s = a.s * fa + b.s * fb;
    r.w = __builtin_fmaf(a.s, da, a.w) * fa + __builtin_fmaf(b.s, db, b.w) * fb;
    return r;
}

template <int STEP>
__device__ __forceinline__ Stats join_step(const Stats &v, float c) {
    return join(v, Stats{partner<STEP>(v.m), partner<STEP>(v.s), partner<STEP>(v.w)}, c);
}
__device__ __forceinline__ Stats join_lanes(Stats v, float c) {
    v = join_step<0>(v, c);
    v = join_step<1>(v, c);
    v = join_step<2>(v, c);
    v = join_step<3>(v, c);
    v = join_step<4>(v, c);
    return join_step<5>(v, c);
}

// The n largest keys a wave has seen, largest in lane 0.  A key is the
// logit's order key over the complement of its column, so a larger logit, and
// among equals the lower column, comes first, in whatever order keys arrive.
struct Best {
    uint64_t list;      // lane i: the i-th largest (0: none yet)
    uint64_t last;      // a key must be above this to enter: the n-th largest, or a lower bound of it
};

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
}

// key into the sorted list: the lanes below its place move up by one
__device__ __forceinline__ void insert(Best &b, uint64_t key, int n, int lane) {
    const int at = __builtin_popcountll(__ballot(b.list > key));
    const uint32_t lo = dpp_mov<0x138>((uint32_t)b.list);              // wave_shr:1
    const uint32_t hi = dpp_mov<0x138>((uint32_t)(b.list >> 32));
    const uint64_t up = ((uint64_t)hi << 32) | lo;
    b.list = lane < at ? b.list : lane == at ? key : up;
    const uint64_t nth = readlane64(b.list, n - 1);
    b.last = nth > b.last ? nth : b.last;
}

// every lane's key that beats the n-th so far
__device__ __forceinline__ void offer(Best &b, uint64_t key, int n, int lane) {
    for (uint64_t m = __ballot(key > b.last); m; m &= m - 1) {
        const uint64_t k = readlane64(key, __builtin_ctzll(m));
        if (k > b.last) insert(b, k, n, lane);
    }
}

// Raises the bar of an empty list to the n-th largest of one value per lane
// (each lane holding a key with that order key at least), so that a first
// batch of many values costs about n insertions instead of n log(values / n).
// The value's upper 16 bits are found by bisection, one ballot a bit.
__device__ __forceinline__ void raise(Best &b, uint32_t order, int n) {
    uint32_t bar = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t t = bar | (1u << bit);
        if (__builtin_popcountll(__ballot(order >= t)) >= n) bar = t;
    }
    if (bar) b.last = ((uint64_t)bar << 32) - 1;
}

// the n largest of `count` keys (0: none) in memory
__device__ __forceinline__ Best best_of(const uint64_t *keys, int count, int n, int lane) {
    Best b{0, 0};
    uint32_t order = 0;
    for (int i = lane; i < count; i += 64) {
        const uint32_t o = (uint32_t)(keys[i] >> 32);
        order = o > order ? o : order;
    }
    raise(b, order, n);
    for (int i = 0; i < count; i += 64) offer(b, i + lane < count ? keys[i + lane] : 0, n, lane);
    return b;
}

__device__ __forceinline__ uint64_t logit_key(float x, int64_t col) {
    return ((uint64_t)order_key(x) << 32) | (uint32_t)~(uint32_t)col;
}

// N logits of every lane into its running statistics and, with TOP, the
// wave's best list.  One new maximum and one rescaling for the N together, so
// the maximum is exact and no term is positive.  Logit i of a lane is in
// column col + (i / V) * step + i % V; columns from hi on hold -Inf.
template <int N, int V, bool TOP>
__device__ __forceinline__ void take(Stats &v, Best &best, const float *x, float c, int64_t col, int64_t step, int64_t hi,
                                     int n, int lane) {
    float g = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) g = __builtin_fmaxf(g, x[i]);
    const float m = __builtin_fmaxf(v.m, g);
    const float d = __builtin_fmaxf((v.m - m) * c, -1000.0f);
    const float f = __builtin_amdgcn_exp2f(d);
    v.w = __builtin_fmaf(v.s, d, v.w) * f;
    v.s *= f;
    v.m = m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float u = (x[i] - m) * c;
        const float e = __builtin_amdgcn_exp2f(u);
        v.s += e;
        v.w = __builtin_fmaf(e, __builtin_fmaxf(u, -1000.0f), v.w);     // 0 * -Inf stays 0; a NaN is in s
    }
    if constexpr (TOP) {
        // an empty list's bar is 0, the key of a NaN, which no g is below
        if (__ballot(!(g < order_value((uint32_t)(best.last >> 32))))) {
            if (best.last == 0) raise(best, col < hi ? order_key(g) : 0u, n);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!__ballot(!(x[i] < order_value((uint32_t)(best.last >> 32))))) continue;
                const int64_t at = col + i / V * step + i % V;
                offer(best, at < hi ? logit_key(x[i], at) : 0, n, lane);
            }
        }
    }
}

// Writes a row's results; the whole wave, with the joined statistics.  What
// divides by the temperature is computed in fp64 and rounded once: a row has
// few such values, and the quotients of two logits would otherwise each
// round at their own size instead of that of their distance.
template <class E>
__device__ __forceinline__ void finish_row(const LogprobsArgs &a, int64_t t, const Stats &v, uint64_t list, int lane) {
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    const bool none = v.s == 0.0f;                       // every logit -Inf
    float top = none ? -__builtin_inff() : v.m;
    if (v.s != v.s && !(v.m > -kLowest)) top = v.s;      // a NaN among the logits
    const float log_sum = none ? __builtin_nanf("") : logf(v.s);
    if (lane == 0) {
        const int64_t target = a.targets[t];
        float lp = 0.0f;
        if (target >= 0 && target < a.V)
            lp = (float)(((double)Elem<E>::get(row[target]) - top) / a.temperature - log_sum);
        a.logprobs[t] = lp;
        a.entropy[t] = none ? __builtin_nanf("") : log_sum - v.w / v.s * kLn2;
        a.stats[2 * t] = (float)(top / a.temperature);
        a.stats[2 * t + 1] = log_sum;
    }
    if (lane < a.top) {
        a.top_ids[t * a.top + lane] = (uint32_t)~(uint32_t)list;
        const double x = order_value((uint32_t)(list >> 32));
        a.top_logprobs[t * a.top + lane] = (float)((x - top) / a.temperature - log_sum);
    }
}

// Partial results of a slice of a row in the workspace: [T][slices] of Stats
// padded to 16 bytes, then [T][slices][top] keys.
__device__ __forceinline__ float4 *part_stats(const LogprobsArgs &a) { return static_cast<float4 *>(a.workspace); }
__device__ __forceinline__ uint64_t *part_keys(const LogprobsArgs &a) {
    return reinterpret_cast<uint64_t *>(part_stats(a) + a.T * a.slices);
}

// One pass over a slice of a row: running maximum, sum and weighted sum per
// lane, joined over the block.
template <class E, bool TOP, int BLOCK>
__global__ __launch_bounds__(BLOCK) void logprobs_kernel(const LogprobsArgs a) {
    constexpr int kV = Elem<E>::kVec, kWaves = BLOCK / 64;
    __shared__ Stats parts[kWaves];
    __shared__ uint64_t keys[TOP ? kWaves * kLogprobsMaxTop : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x / a.slices;
    const int slice = (int)((int64_t)blockIdx.x - t * a.slices);
    const int64_t lo = slice * a.slice;
    const int64_t hi = lo + a.slice < a.V ? lo + a.slice : a.V;
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    const float c = a.scale;
    Stats v{kLowest, 0.0f, 0.0f};
    Best best{0, 0};

    constexpr int kStep = BLOCK * kV;
    int64_t col = lo + threadIdx.x * kV;
    int64_t base = lo;                               // the block's position, the same in all lanes
    for (; base + kUnroll * kStep <= hi; base += kUnroll * kStep, col += kUnroll * kStep) {
        v4u r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) r[u] = load16(row + col + u * kStep);
        float x[kUnroll * kV];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) Elem<E>::unpack(r[u], x + u * kV);
        take<kUnroll * kV, kV, TOP>(v, best, x, c, col, kStep, hi, a.top, lane);
    }
    for (; base < hi; base += kStep, col += kStep) {
        float x[kV];
        const int64_t n = hi - col;
        if (n >= kV) {
            Elem<E>::unpack(load16(row + col), x);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = i < n ? Elem<E>::get(row[col + i]) : -__builtin_inff();
        }
        take<kV, kV, TOP>(v, best, x, c, col, 0, hi, a.top, lane);
    }

    v = join_lanes(v, c);
    if (lane == 0) parts[wave] = v;
    if constexpr (TOP) {
        if (lane < a.top) keys[wave * a.top + lane] = best.list;
    }
    __syncthreads();
    if (wave != 0) return;
    v = join_lanes(lane < kWaves ? parts[lane] : Stats{kLowest, 0.0f, 0.0f}, c);
    if constexpr (TOP) best = best_of(keys, kWaves * a.top, a.top, lane);
    if (a.slices == 1) {
        finish_row<E>(a, t, v, best.list, lane);
    } else {
        if (lane == 0) part_stats(a)[blockIdx.x] = make_float4(v.m, v.s, v.w, 0.0f);
        if constexpr (TOP) {
            if (lane < a.top) part_keys(a)[(int64_t)blockIdx.x * a.top + lane] = best.list;
        }
    }
}

// Joins the slices of a row, one wave a row.
template <class E>
__global__ __launch_bounds__(64) void logprobs_join_kernel(const LogprobsArgs a) {
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const float c = a.scale;
    Stats v{kLowest, 0.0f, 0.0f};
    for (int s = lane; s < a.slices; s += 64) {
        const float4 p = part_stats(a)[t * a.slices + s];
        v = join(v, Stats{p.x, p.y, p.z}, c);
    }
    v = join_lanes(v, c);
    Best best{0, 0};
    if (a.top) {
        const int n = a.slices * a.top;
        best = best_of(part_keys(a) + t * n, n, a.top, lane);
    }
    finish_row<E>(a, t, v, best.list, lane);
}

// d logits = (g (1[target] - p) - h p (log p + H)) / temp with g, h the
// gradients of log-probability and entropy, log p = x / temp - m - log_sum.
// One read and one write of the logits; in place is fine (a thread writes
// what it alone has read).
template <class E>
__global__ __launch_bounds__(kBlock) void logprobs_backward_kernel(const LogprobsArgs a) {
    constexpr int kV = Elem<E>::kVec;
    const int64_t t = (int64_t)blockIdx.x / a.slices;
    const int slice = (int)((int64_t)blockIdx.x - t * a.slices);
    const int64_t lo = slice * a.slice;
    const int64_t hi = lo + a.slice < a.V ? lo + a.slice : a.V;
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    E *out = static_cast<E *>(a.dx) + t * a.ld_out;
    const int64_t target = a.targets[t];
    const bool real = target >= 0 && target < a.V;
    const float g = real && a.d_logprobs ? a.d_logprobs[t] : 0.0f;
    const float h = a.d_entropy ? a.d_entropy[t] : 0.0f;
    const float H = h != 0.0f ? a.entropy[t] : 0.0f;
    const float m = a.stats[2 * t], log_sum = a.stats[2 * t + 1];
    const float inv = a.inv, inv_low = a.inv_low;                            // 1 / temp = inv + inv_low
    const float c0 = -(g + h * H) * inv, c1 = -h * inv, at_target = g * inv;
    for (int64_t col = lo + threadIdx.x * kV; col < hi; col += kBlock * kV) {
        float x[kV];
        const int64_t n = hi - col;
        if (n >= kV) {
            Elem<E>::unpack(load16(row + col), x);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = i < n ? Elem<E>::get(row[col + i]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float logp = __builtin_fmaxf(__builtin_fmaf(x[i], inv, __builtin_fmaf(x[i], inv_low, -m)) - log_sum, -1000.0f);
            const float p = __builtin_amdgcn_exp2f(logp * kLog2E);
            float d = p * __builtin_fmaf(c1, logp, c0);
            if (col + i == target) d += at_target;
            x[i] = d;
        }
        if (n >= kV) {
            store16(out + col, Elem<E>::pack(x));
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i < n) out[col + i] = Elem<E>::put(x[i]);
        }
    }
}

// Slices of a row: one where the rows alone give every compute unit a block,
// else enough for four blocks each, of at least 4096 logits.
int slices_of(int64_t T, int64_t V, int cus) {
    if (T >= cus) return 1;
    const int64_t want = ceil_div((int64_t)cus * 4, T), most = ceil_div(V, 4096);
    return (int)(want < most ? want : most);
}

template <class E, bool TOP>
void start(const LogprobsArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.T * a.slices);
    if (a.slice > 16384) logprobs_kernel<E, TOP, kWide><<<grid, kWide, 0, stream>>>(a);
    else logprobs_kernel<E, TOP, kBlock><<<grid, kBlock, 0, stream>>>(a);
    if (a.slices > 1) logprobs_join_kernel<E><<<(unsigned)a.T, 64, 0, stream>>>(a);
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t T, int64_t V, int top, int cus) {
    const int s = slices_of(T, V, cus);
    return s == 1 ? 0 : T * s * (16 + 8 * (int64_t)top);
}

hipError_t launch_logprobs(LogprobsArgs a, bool bf16, size_t workspace_bytes, hipStream_t stream) {
    const int cus = device_cu_count();
    a.scale = (float)(1.4426950408889634 / a.temperature);
    a.slices = slices_of(a.T, a.V, cus);
    if (!a.workspace || (int64_t)workspace_bytes < logprobs_workspace_bytes(a.T, a.V, a.top, cus)) a.slices = 1;
    a.slice = ceil_div(ceil_div(a.V, a.slices), 8) * 8;
    if (bf16) {
        if (a.top) start<uint16_t, true>(a, stream);
        else start<uint16_t, false>(a, stream);
    } else {
        if (a.top) start<float, true>(a, stream);
        else start<float, false>(a, stream);
    }
    return hipGetLastError();
}

hipError_t launch_logprobs_backward(LogprobsArgs a, bool bf16, hipStream_t stream) {
    a.inv = (float)(1.0 / a.temperature);
    a.inv_low = (float)(1.0 / a.temperature - a.inv);
    a.slice = 4 * kBlock * (bf16 ? 8 : 4);
    a.slices = (int)ceil_div(a.V, a.slice);
    const unsigned grid = (unsigned)(a.T * a.slices);
    if (bf16) logprobs_backward_kernel<uint16_t><<<grid, kBlock, 0, stream>>>(a);
    else logprobs_backward_kernel<float><<<grid, kBlock, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace mx
