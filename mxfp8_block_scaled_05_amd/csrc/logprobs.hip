// Log-probabilities of given tokens, entropy and the likeliest tokens of rows
// of logits, and the gradient of the first two.
#include <type_traits>

#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;         // threads of the gradient's blocks
constexpr int kUnroll = 4;          // 16-byte loads of a thread in flight
constexpr float kLowest = -3.402823466e38f;
// From here on different fp32 logits have z at least 2^7 apart: e^-128 is 0.
constexpr float kFar = 0x1p31f;

// z = x / temperature rounded to fp32; finite logits stay finite
__device__ __forceinline__ float scaled(float x, double inv_temperature) {
    const double z = x * inv_temperature;
    return __builtin_isinf(x) ? x : z > -kLowest ? -kLowest : z < kLowest ? kLowest : (float)z;
}

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
    int have;           // entries of the list, at most n
    uint64_t *room;     // LDS of the wave: 64 keys
};

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ void new_bar(Best &b, int n) {
    const uint64_t nth = readlane64(b.list, n - 1);
    b.last = nth > b.last ? nth : b.last;
}

// key into the sorted list: the lanes below its place move up by one
__device__ __forceinline__ void insert(Best &b, uint64_t key, int n, int lane) {
    const int at = __builtin_popcountll(__ballot(b.list > key));
    const uint32_t lo = dpp_mov<0x138>((uint32_t)b.list);              // wave_shr:1
    const uint32_t hi = dpp_mov<0x138>((uint32_t)(b.list >> 32));
    const uint64_t up = ((uint64_t)hi << 32) | lo;
    b.list = lane < at ? b.list : lane == at ? key : up;
    b.have = b.have < n ? b.have + 1 : n;
    new_bar(b, n);
}

// every lane's key that beats the n-th so far, one after another
__device__ __forceinline__ void offer(Best &b, uint64_t key, int n, int lane) {
    for (uint64_t m = __ballot(key > b.last); m; m &= m - 1) {
        const uint64_t k = readlane64(key, __builtin_ctzll(m));
        if (k > b.last) insert(b, k, n, lane);
    }
}

// Many keys at once: those above the bar are laid down in the wave's room
// beside the list (gather), and all of them ranked together (settle), each
// lane counting the keys above its own.  An insertion is a chain of about 25
// dependent steps; ranking 40 keys costs as much as four of them.
__device__ __forceinline__ int gather_begin(const Best &b, int lane) {
    if (lane < b.have) b.room[lane] = b.list;
    return b.have;
}
__device__ __forceinline__ void settle(Best &b, int held, int n, int lane) {
    wave_sync();
    const uint64_t mine = lane < held ? b.room[lane] : 0;
    int rank = 0;
    for (int j = 0; j < held; ++j) rank += readlane64(mine, j) > mine ? 1 : 0;
    wave_sync();
    if (lane < held) b.room[rank] = mine;                // keys differ, so ranks do
    wave_sync();
    b.have = held < n ? held : n;
    b.list = lane < b.have ? b.room[lane] : 0;
    new_bar(b, n);
}
__device__ __forceinline__ void gather(Best &b, int &held, uint64_t key, int n, int lane) {
    uint64_t m = __ballot(key > b.last);
    if (!m) return;
    if (held + __builtin_popcountll(m) > 64) {           // full: what is there first
        settle(b, held, n, lane);
        held = b.have;
        m = __ballot(key > b.last);
        if (held + __builtin_popcountll(m) > 64) {
            offer(b, key, n, lane);
            held = gather_begin(b, lane);
            return;
        }
    }
    const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    if ((m >> lane) & 1) b.room[held + below] = key;
    held += __builtin_popcountll(m);
}

// A bar that n of the wave's values reach (N a lane): the n-th largest, its
// upper 16 bits, by bisection.
template <int N>
__device__ __forceinline__ uint32_t bar_of(const uint32_t (&order)[N], int n) {
    uint32_t bar = 0;
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t t = bar | (1u << bit);
        int count = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) count += __builtin_popcountll(__ballot(order[i] >= t));
        if (count >= n) bar = t;
    }
    return bar;
}
// the last key below every key of order `bar` or more
__device__ __forceinline__ uint64_t below_bar(uint32_t bar) { return bar ? ((uint64_t)bar << 32) - 1 : 0; }

// The n largest of `count` keys (0: none) in memory that are above last.  With
// no such bar known (last = 0) the first keys give one.
template <int AHEAD>
__device__ __forceinline__ Best best_of(const uint64_t *keys, int count, int n, uint64_t last, uint64_t *room, int lane) {
    Best b{0, last, 0, room};
    int held = 0;
    for (int i0 = 0; i0 < count; i0 += 64 * AHEAD) {
        uint64_t k[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int i = i0 + u * 64 + lane;
            k[u] = keys[i < count ? i : 0];
            if (i >= count) k[u] = 0;
        }
        if (i0 == 0 && last == 0) {
            uint32_t order[1] = {0};
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) order[0] = (uint32_t)(k[u] >> 32) > order[0] ? (uint32_t)(k[u] >> 32) : order[0];
            b.last = below_bar(bar_of(order, n));
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u * 64 < count) gather(b, held, k[u], n, lane);
    }
    settle(b, held, n, lane);
    return b;
}

// Unsigned order of a logit among a row's best: a NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t logit_order(float x) { return x != x ? 0xFFFFFFFFu : order_key(x + 0.0f); }
__device__ __forceinline__ uint64_t logit_key(float x, int64_t col) {
    return ((uint64_t)logit_order(x) << 32) | (uint32_t)~(uint32_t)col;
}

// N logits of every lane into its running statistics; returns their maximum.
// One new maximum and one rescaling for the N together, so the maximum is
// exact and no term is positive.
template <int N>
__device__ __forceinline__ float take(Stats &v, const float *x, float c) {
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
    return g;
}

// n logits of type E at p (all of kV, or the first n and -Inf)
template <class E>
__device__ __forceinline__ void load_logits(const E *p, int64_t n, float *x) {
    constexpr int kV = Elem<E>::kVec;
    if (n >= kV) {
        Elem<E>::unpack(load16(p), x);
    } else if (n > 0) {
        load_head<kV>(p, (int)n, -__builtin_inff(), x);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = -__builtin_inff();
    }
}

// The target of a row and its logit, asked for at the start of a kernel: two
// loads in a row, which would otherwise wait at its end.
struct Target {
    bool real;
    float x;
};
template <class E>
__device__ __forceinline__ Target load_target(const LogprobsArgs &a, int64_t t) {
    const int64_t v = a.targets[t];
    const bool real = v >= 0 && v < a.V;
    return {real, Elem<E>::get(static_cast<const E *>(a.x)[t * a.ld + (real ? v : 0)])};
}

// Writes a row's results; the whole wave, with the joined statistics.  What
// divides by the temperature is computed in fp64 and rounded once: a row has
// few such values, and the quotients of two logits would otherwise each
// round at their own size instead of that of their distance.
__device__ __forceinline__ void finish_row(const LogprobsArgs &a, int64_t t, const Stats &v, const Target &target,
                                           uint64_t list, int lane) {
    const bool none = v.s == 0.0f;                       // every logit -Inf
    float top = none ? -__builtin_inff() : v.m;
    if (v.s != v.s && !(v.m > -kLowest)) top = v.s;      // a NaN among the logits
    const float log_sum = none ? __builtin_nanf("") : logf(v.s);
    if (lane == 0) {
        a.logprobs[t] = target.real ? (float)(((double)target.x - top) * a.inv_temperature - log_sum) : 0.0f;
        a.entropy[t] = none ? __builtin_nanf("") : log_sum - v.w / v.s * kLn2;
        // L against the rounded m, so that the gradient's z - m - L loses nothing by that rounding
        const float m = scaled(top, a.inv_temperature);
        a.stats[2 * t] = m;
        a.stats[2 * t + 1] = __builtin_fabsf(m) < kFar ? (float)(log_sum + (top * a.inv_temperature - m)) : log_sum;
    }
    if (lane < a.top) {
        a.top_ids[t * a.top + lane] = (uint32_t)~(uint32_t)list;
        const double x = order_value((uint32_t)(list >> 32));
        a.top_logprobs[t * a.top + lane] = (float)((x - top) * a.inv_temperature - log_sum);
    }
}

// Partial results of a slice of a row in the workspace: [T][slices] of Stats
// padded to 16 bytes, then [T][slices][top] keys.
__device__ __forceinline__ float4 *part_stats(const LogprobsArgs &a) { return static_cast<float4 *>(a.workspace); }
__device__ __forceinline__ uint64_t *part_keys(const LogprobsArgs &a) {
    return reinterpret_cast<uint64_t *>(part_stats(a) + a.T * a.slices);
}

// One pass over a slice of a row: running maximum, sum and weighted sum per
// lane, joined over the block.  2048 rows of 131072 bf16 take 88 us, 6.1 TB/s
// (only reading them 80): HBM and the vector ALU (9.2 instructions a logit, busy
// nearly all of the time) are both at their limits; one row of 131072 5.1 us.
// ONCE: the logits are larger than the last-level cache and are read past it
// (91.5 us if not; the call and its gradient 263 us instead of 293).
//
// The best n: the pass keeps each thread's largest logit only.  n threads'
// largest reach the n-th largest of them, so no logit below that bar is among
// the best, and few threads hold one above it: their logits alone are looked
// at again (n / BLOCK of the row), those above the bar gathered and ranked.
// 2048 rows of 131072 bf16 with n = 5: 107 us (a list kept sorted during the
// pass: 182); one row with n = 20: 12.6 us with the join (22).
template <class E, bool TOP, int BLOCK, bool ONCE>
__global__ __launch_bounds__(BLOCK) void logprobs_kernel(const LogprobsArgs a) {
    constexpr int kV = Elem<E>::kVec, kWaves = BLOCK / 64;
    __shared__ Stats parts[kWaves];
    __shared__ uint64_t keys[TOP ? kWaves * kLogprobsMaxTop : 1];
    __shared__ uint64_t room[TOP ? kWaves : 1][64];
    __shared__ uint32_t largest[TOP ? BLOCK : 1];
    __shared__ uint32_t shared_bar;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x / a.slices;
    const int slice = (int)((int64_t)blockIdx.x - t * a.slices);
    const int64_t lo = slice * a.slice;
    const int64_t hi = lo + a.slice < a.V ? lo + a.slice : a.V;
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    const float c = a.scale;
    Target target{false, 0.0f};
    if (wave == 0 && a.slices == 1) target = load_target<E>(a, t);
    Stats v{kLowest, 0.0f, 0.0f};
    float most = -__builtin_inff();

    constexpr int kStep = BLOCK * kV;
    int64_t col = lo + threadIdx.x * kV;
    int64_t base = lo;                               // the block's position, the same in all lanes
    auto steps = [&](auto unroll) {                  // that many loads in flight, and one rescaling for them
        constexpr int U = decltype(unroll)::value;
        for (; base + U * kStep <= hi; base += U * kStep, col += U * kStep) {
            v4u r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = load16<ONCE>(row + col + u * kStep);
            float x[U * kV];
#pragma unroll
            for (int u = 0; u < U; ++u) Elem<E>::unpack(r[u], x + u * kV);
            most = __builtin_fmaxf(most, take<U * kV>(v, x, c));
        }
    };
    steps(std::integral_constant<int, kUnroll>());
    steps(std::integral_constant<int, kUnroll / 2>());
    for (; base < hi; base += kStep, col += kStep) {
        float x[kV];
        load_logits(row + col, hi - col, x);
        most = __builtin_fmaxf(most, take<kV>(v, x, c));
    }

    v = join_lanes(v, c);
    if (lane == 0) parts[wave] = v;
    const uint32_t mine = logit_order(most);
    if constexpr (TOP) largest[threadIdx.x] = mine;
    __syncthreads();
    if constexpr (TOP) {
        if (wave == 0) {
            uint32_t order[kWaves];
#pragma unroll
            for (int i = 0; i < kWaves; ++i) order[i] = largest[i * 64 + lane];
            const uint32_t bar = bar_of(order, a.top);
            if (lane == 0) shared_bar = bar;
        }
        __syncthreads();
        const uint64_t last = below_bar(shared_bar);
        Best best{0, last, 0, room[wave]};
        int held = 0;
        // 2^shift lanes look at the pieces of one thread, `at` the first column of piece 0
        const int pieces = (int)((hi - lo + kStep - 1) / kStep);
        int shift = 0;
        while (shift < 6 && (1 << shift) < pieces) ++shift;
        for (uint64_t m = __ballot(mine >= shared_bar); m;) {
            int from = -1;
            for (int q = 0; q < 64 >> shift && m; ++q, m &= m - 1)
                if (lane >> shift == q) from = __builtin_ctzll(m);
            for (int piece = 0; piece < pieces; piece += 64) {
                const int mypiece = piece + (lane & ((1 << shift) - 1));
                const int64_t at = lo + (wave * 64 + from) * kV + (int64_t)mypiece * kStep;
                const int64_t n = from >= 0 ? hi - at : 0;
                float x[kV];
                load_logits(row + at, n, x);
#pragma unroll
                for (int i = 0; i < kV; ++i) gather(best, held, i < n ? logit_key(x[i], at + i) : 0, a.top, lane);
            }
        }
        wave_sync();
        if (best.have || held > a.top) settle(best, held, a.top, lane);
        else best.list = lane < held ? room[wave][lane] : 0;            // in any order: they are ranked below
        if (lane < a.top) keys[wave * a.top + lane] = best.list;
        __syncthreads();
        if (wave != 0) return;
        best = best_of<4>(keys, kWaves * a.top, a.top, last, room[0], lane);
        v = join_lanes(lane < kWaves ? parts[lane] : Stats{kLowest, 0.0f, 0.0f}, c);
        if (a.slices == 1) {
            finish_row(a, t, v, target, best.list, lane);
        } else {
            if (lane == 0) part_stats(a)[blockIdx.x] = make_float4(v.m, v.s, v.w, 0.0f);
            if (lane < a.top) part_keys(a)[(int64_t)blockIdx.x * a.top + lane] = best.list;
        }
    } else {
        if (wave != 0) return;
        v = join_lanes(lane < kWaves ? parts[lane] : Stats{kLowest, 0.0f, 0.0f}, c);
        if (a.slices == 1) finish_row(a, t, v, target, 0, lane);
        else if (lane == 0) part_stats(a)[blockIdx.x] = make_float4(v.m, v.s, v.w, 0.0f);
    }
}

// Joins the slices of a row, one wave a row.
template <class E>
__global__ __launch_bounds__(64) void logprobs_join_kernel(const LogprobsArgs a) {
    __shared__ uint64_t room[64];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const Target target = load_target<E>(a, t);
    const float c = a.scale;
    Stats v{kLowest, 0.0f, 0.0f};
    for (int s = lane; s < a.slices; s += 64) {
        const float4 p = part_stats(a)[t * a.slices + s];
        v = join(v, Stats{p.x, p.y, p.z}, c);
    }
    v = join_lanes(v, c);
    uint64_t list = 0;
    if (a.top) {
        const int n = a.slices * a.top;
        const uint64_t *keys = part_keys(a) + t * n;
        list = best_of<12>(keys, n, a.top, 0, room, lane).list;
    }
    finish_row(a, t, v, target, list, lane);
}

// A row's distances z - m as x (by + by_low) - from, and a bound of log p.
struct Line {
    float by, by_low, from, most;
};

// The line of a row with |m| >= kFar.  A distance there is 0 or far below -128
// and what x loses in z's rounding more than either, so the line starts at the
// smallest logit whose z rounds to m, is steep enough to take every lower one
// (2^-24 of it away at least) to p = 0, and log p ends at -L.
__device__ __forceinline__ Line far_line(const LogprobsArgs &a, float m, float log_sum) {
    const double at = (double)m * a.temperature;                 // within 2 steps of fp32 of that logit
    float x = at > -kLowest ? -kLowest : at < kLowest || m <= kLowest ? kLowest : (float)at;
    const uint32_t down = m < 0.0f ? 1u : -1u;
    for (int i = 0; i < 3; ++i) {
        const float lower = __uint_as_float(__float_as_uint(x) + down);
        if (lower >= kLowest && scaled(lower, a.inv_temperature) == m) x = lower;
    }
    for (int i = 0; i < 3; ++i)
        if (scaled(x, a.inv_temperature) < m) x = __uint_as_float(__float_as_uint(x) - down);
    const int exponent = (int)((__float_as_uint(x) >> 23) & 255) - 127;
    const float by = __builtin_ldexpf(1.0f, 40 - exponent);      // x * by: 2^40 to 2^41
    return {by, 0.0f, x * by, -log_sum};
}

// d logits = (g (1[target] - p) - h p (log p + H)) / temp with g, h the
// gradients of log-probability and entropy, log p = x / temp - m - log_sum.
// One read and one write of the logits; in place is fine (a thread writes
// what it alone has read).  2048 rows of 131072 bf16 take 174 us, 6.2 TB/s (a
// copy past the caches 165).  ONCE: what is read and written (in place: the
// logits alone) is larger than the last-level cache and goes past it (187 us
// if not; but 511 rows of 100003 fp32 written, scored and overwritten in place,
// which fit, would take 185 us instead of 167).  A row of 9000 in two blocks of equal length 53
// us, cut at 8192 72 us (8000 rows).
template <class E, int BLOCK, bool ONCE>
__global__ __launch_bounds__(BLOCK) void logprobs_backward_kernel(const LogprobsArgs a) {
    constexpr int kV = Elem<E>::kVec, kStep = BLOCK * kV;
    const int64_t t = (int64_t)blockIdx.x / a.slices;
    const int slice = (int)((int64_t)blockIdx.x - t * a.slices);
    const int64_t lo = slice * a.slice;
    const int64_t hi = lo + a.slice < a.V ? lo + a.slice : a.V;
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    E *out = static_cast<E *>(a.dx) + t * a.ld_out;
    const int64_t col = lo + threadIdx.x * kV;
    v4u r[kUnroll];                                  // a thread's whole share, before anything is written
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (hi - col - u * kStep >= kV) r[u] = load16<ONCE>(row + col + u * kStep);
    const int64_t target = a.targets[t];
    const bool real = target >= 0 && target < a.V;
    const float g = real && a.d_logprobs ? a.d_logprobs[t] : 0.0f;
    const float h = a.d_entropy ? a.d_entropy[t] : 0.0f;
    const float H = h != 0.0f ? a.entropy[t] : 0.0f;
    const float m = a.stats[2 * t], log_sum = a.stats[2 * t + 1];
    const float inv = a.inv, inv_low = a.inv_low;                            // 1 / temp = inv + inv_low
    // L is NaN in a row without statistics (a NaN or +Inf in it, or nothing above -Inf): c0 takes that to every
    // column, since the lower limit of log p, which stands for -Inf columns, drops a NaN
    const float c0 = -(g + h * H) * inv + (log_sum - log_sum), c1 = -h * inv, at_target = g * inv;
    Line line{inv, inv_low, m, 1000.0f};
    if (__builtin_fabsf(m) >= kFar) line = far_line(a, m, log_sum);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t at = col + u * kStep, n = hi - at;
        if (n <= 0) break;
        float x[kV];
        if (n >= kV) Elem<E>::unpack(r[u], x);
        else load_head<kV>(row + at, (int)n, 0.0f, x);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            // one rounding of x * by - from, which is about as large as the distance: z itself is never rounded
            const float z = __builtin_fmaf(x[i], line.by_low, __builtin_fmaf(x[i], line.by, -line.from));
            const float logp = __builtin_amdgcn_fmed3f(z - log_sum, -1000.0f, line.most);
            const float p = __builtin_amdgcn_exp2f(logp * kLog2E);
            float d = p * __builtin_fmaf(c1, logp, c0);
            if (at + i == target) d += at_target;
            x[i] = d;
        }
        if (n >= kV) {
            store16<ONCE>(out + at, Elem<E>::pack(x));
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i < n) out[at + i] = Elem<E>::put(x[i]);
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

// Threads of a block, from the length of its slice, the rows and whether it
// looks for the best n (whose steps are short and in sequence: smaller blocks
// let another block of the unit stream meanwhile).  us with 64 / 128 / 256 /
// 512 / 1024 threads:
//   8000 rows of 1001 bf16            9.7 / 12.1 / 18.2 / 30.6 / 56.8
//   the same with n = 5              15.8 / 20.8 / 32.6 / 82.4 / 224
//   8000 rows of 8001 bf16, n = 5    38.9 / 36.7 / 47.6 / 90.8 / 230
//   300 rows of 16001 bf16            8.7 /  7.6 /  6.2 /  6.3 /  7.1
//   2600 rows of 50001 bf16          50.7 / 50.7 / 48.9 / 51.4 / 59.7
//   1340 rows of 100003 fp32          105 /  104 /  104 / 98.6 / 96.2
//   1340 rows of 100003 bf16, n = 5  91.7 / 68.1 / 59.3 / 57.4 / 91.3
template <class E, bool TOP, bool ONCE>
void start(const LogprobsArgs &a, int cus, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.T * a.slices);
    const bool many = a.T >= 4 * cus;
    constexpr int wide = TOP ? 512 : 1024;
    if (many && a.slice <= 2048) logprobs_kernel<E, TOP, 64, ONCE><<<grid, 64, 0, stream>>>(a);
    else if (many && a.slice <= 8192) logprobs_kernel<E, TOP, 128, ONCE><<<grid, 128, 0, stream>>>(a);
    else if (a.slice <= (TOP ? 32768 : 65536)) logprobs_kernel<E, TOP, 256, ONCE><<<grid, 256, 0, stream>>>(a);
    else logprobs_kernel<E, TOP, wide, ONCE><<<grid, wide, 0, stream>>>(a);
    if (a.slices > 1) logprobs_join_kernel<E><<<(unsigned)a.T, 64, 0, stream>>>(a);
}
template <class E>
void start(const LogprobsArgs &a, int cus, hipStream_t stream) {
    const bool once = a.T * a.V * (int64_t)sizeof(E) > kLastLevelBytes;
    if (a.top) once ? start<E, true, true>(a, cus, stream) : start<E, true, false>(a, cus, stream);
    else once ? start<E, false, true>(a, cus, stream) : start<E, false, false>(a, cus, stream);
}
template <class E, int BLOCK>
void start_backward(const LogprobsArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.T * a.slices);
    const int64_t bytes = a.T * a.V * (int64_t)sizeof(E);
    if ((a.x == a.dx ? bytes : 2 * bytes) > kLastLevelBytes)
        logprobs_backward_kernel<E, BLOCK, true><<<grid, BLOCK, 0, stream>>>(a);
    else
        logprobs_backward_kernel<E, BLOCK, false><<<grid, BLOCK, 0, stream>>>(a);
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t T, int64_t V, int top, int cus) {
    const int s = slices_of(T, V, cus);
    return s == 1 ? 0 : T * s * (16 + 8 * (int64_t)top);
}

hipError_t launch_logprobs(LogprobsArgs a, bool bf16, size_t workspace_bytes, hipStream_t stream) {
    const int cus = device_cu_count();
    a.inv_temperature = 1.0 / a.temperature;
    a.scale = (float)(1.4426950408889634 * a.inv_temperature);
    a.slices = slices_of(a.T, a.V, cus);
    if (!a.workspace || (int64_t)workspace_bytes < logprobs_workspace_bytes(a.T, a.V, a.top, cus)) a.slices = 1;
    a.slice = ceil_div(ceil_div(a.V, a.slices), 8) * 8;
    if (bf16) start<uint16_t>(a, cus, stream);
    else start<float>(a, cus, stream);
    return hipGetLastError();
}

hipError_t launch_logprobs_backward(LogprobsArgs a, bool bf16, hipStream_t stream) {
    a.inv_temperature = 1.0 / a.temperature;
    a.inv = (float)a.inv_temperature;
    a.inv_low = (float)(a.inv_temperature - a.inv);
    // blocks of kUnroll 16-byte pieces a thread at most, a row's blocks of about the same length
    const int vec = bf16 ? 8 : 4;
    const bool narrow = a.V <= kUnroll * vec * 64;
    const int64_t most = kUnroll * vec * (narrow ? 64 : kBlock);
    a.slices = (int)ceil_div(a.V, most);
    a.slice = ceil_div(ceil_div(a.V, a.slices), vec) * vec;
    if (bf16) narrow ? start_backward<uint16_t, 64>(a, stream) : start_backward<uint16_t, kBlock>(a, stream);
    else narrow ? start_backward<float, 64>(a, stream) : start_backward<float, kBlock>(a, stream);
    return hipGetLastError();
}

}  // namespace mx
