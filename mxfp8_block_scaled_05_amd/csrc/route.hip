// Expert routing: the choice of every token's experts and their weights, and
// the gradient of those weights.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;

// NV values of a lane, count of them in the row (the rest become `pad`).  p is
// readable also with count 0.
template <int NV, class E>
__device__ __forceinline__ void load_values(const E *p, int count, float pad, float (&x)[NV]) {
    if constexpr (NV >= Elem<E>::kVec) {
        if (count == NV) {
#pragma unroll
            for (int i = 0; i < NV; i += Elem<E>::kVec) Elem<E>::unpack(load16(p + i), x + i);
            return;
        }
    }
    load_head<NV>(p, count, pad, x);
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, lane, 64);
    const uint32_t hi = (uint32_t)__shfl((int)(uint32_t)(v >> 32), lane, 64);
    return ((uint64_t)hi << 32) | lo;
}

template <int W>
__device__ __forceinline__ uint64_t group_max64(uint64_t v) {
#pragma unroll
    for (int d = 1; d < W; d <<= 1) {
        const uint64_t o = shfl64(v, (int)(threadIdx.x & 63) ^ d);
        v = o > v ? o : v;
    }
    return v;
}

// Lowest lane of the caller's group of L lanes whose bit is set in `b`,
// relative to the group (L if none).
template <int L>
__device__ __forceinline__ int first_lane(uint64_t b, int seg) {
    if constexpr (L == 64) {
        return b ? __builtin_ctzll(b) : L;
    } else {
        const uint32_t m = (uint32_t)(b >> seg) & (uint32_t)((1ull << L) - 1);
        return m ? __builtin_ctz(m) : L;
    }
}

// 1 / (1 + e^-x) for the choice: 2^x and 1/x of the hardware
__device__ __forceinline__ float fast_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2E));
}

// Chosen scores of a token over e^(their largest logit), one a lane, and their
// sum.  Renormalized weights are taken from these where the sum of the scores
// themselves is below kSmallSum: far below, fp32 has no numbers for the scores,
// though for their quotients, and a softmax score is off by 2^-24 of its
// distance from the row's largest logit already before.  (The largest score of a
// softmax is 2^-9 at least, so this is for choices that a bias or groups turn
// away from it, and for sigmoids of nothing but low logits.)  A sigmoid is
// e^x s(-x).  NaN if no logit is above -Inf.
constexpr float kSmallSum = 0x1p-10f;
struct Shares {
    float part, sum;
};
template <int L>
__device__ __forceinline__ Shares shares(float x, bool chosen, bool of_sigmoid) {
    const float most = group_reduce<L>(chosen ? x : -__builtin_inff(), OpMax());
    Shares r;
    r.part = chosen ? exp_neg(x - most) * (of_sigmoid ? sigmoid(-x) : 1.0f) : 0.0f;
    r.sum = group_reduce<L>(r.part, OpAdd());
    return r;
}

// The lanes of one token: group (of experts) g, first expert of the lane and
// how many it holds.
struct LaneExperts {
    int g, first, count;
};
template <int NV>
__device__ __forceinline__ LaneExperts lane_experts(const RouteArgs &a, int l) {
    const int g = l >> a.lanes_shift, q = l & ((1 << a.lanes_shift) - 1);
    LaneExperts e;
    e.g = g;
    e.first = g * a.size + q * NV;
    const int left = a.size - q * NV;
    e.count = g < a.groups ? (left < 0 ? 0 : left > NV ? NV : left) : 0;
    return e;
}

// What the fp64 score of an expert needs besides its logit: for a softmax the
// largest logit of the row and the sum of e^(x - top).
struct Fp64Row {
    double top, total;
};
template <int L, class E>
__device__ __forceinline__ Fp64Row fp64_row(const RouteArgs &a, const E *row, const LaneExperts &ex, float top) {
    Fp64Row r{(double)top, 1.0};
    if (a.sigmoid || a.order_x) return r;
    r.total = 0.0;
#pragma unroll 1
    for (int i = 0; i < ex.count; ++i) r.total += exp((double)Elem<E>::get(row[ex.first + i]) - r.top);
#pragma unroll
    for (int d = 1; d < L; d <<= 1) r.total += __shfl_xor(r.total, d, 64);
    return r;
}
// the value that decides: the biased score, or the logit where that has the same order
__device__ __forceinline__ double fp64_value(const RouteArgs &a, const Fp64Row &r, float x, int id) {
    if (a.order_x) return x + 0.0f;                      // -0 as 0
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - r.top) / r.total;
    return a.bias ? s + (double)a.bias[id] : s;
}

// Whether the lane's group of experts stays, with the groups' scores in fp64.
// Only experts that may be among a group's largest are computed: those above
// `bar` (fp32), one or two a group as a rule.
template <int L, int NV, class E>
__device__ __forceinline__ bool keep_fp64(const RouteArgs &a, const E *row, const LaneExperts &ex, const Fp64Row &r,
                                          const float (&v)[NV], float bar, int lane) {
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) some |= (i < ex.count && !(v[i] < bar)) ? 1u << i : 0u;
    double b1 = -__builtin_inf(), b2 = -__builtin_inf();
    for (; some; some &= some - 1) {
        const int id = ex.first + __builtin_ctz(some);
        const double c = fp64_value(a, r, Elem<E>::get(row[id]), id);
        const double low = c > b1 ? b1 : c;
        b1 = c > b1 ? c : b1;
        b2 = low > b2 ? low : b2;
    }
    for (int d = 1; d < (1 << a.lanes_shift); d <<= 1) {
        const double o1 = __shfl_xor(b1, d, 64), o2 = __shfl_xor(b2, d, 64);
        const double low = o1 < b1 ? o1 : b1, second = o2 > b2 ? o2 : b2;
        b1 = o1 > b1 ? o1 : b1;
        b2 = low > second ? low : second;
    }
    const uint64_t mine = order_key(a.group_top == 2 ? b1 + b2 : b1);
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint64_t o = shfl64(mine, (lane & ~(L - 1)) + (g << a.lanes_shift));
        rank += (o > mine || (o == mine && g < ex.g)) ? 1 : 0;
    }
    return ex.g < a.groups && rank < a.kept;
}

// The whole choice in fp64, for the tokens of a wave of which one has more
// candidates that fp32 cannot order than route_kernel's list holds (many
// equal logits): the same steps on 64-bit keys.  sel[j] of every token gets
// the j-th expert.
template <int L, int NV, class E>
__device__ __forceinline__ void choose_fp64(const RouteArgs &a, const E *row, const LaneExperts &ex, const Fp64Row &r,
                                            bool keep, int lane, int *sel) {
    const int seg = lane & ~(L - 1), l = lane & (L - 1);
    double c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        c[i] = i < ex.count ? fp64_value(a, r, Elem<E>::get(row[ex.first + i]), ex.first + i) : 0.0;
    uint32_t left = keep ? (1u << ex.count) - 1u : 0u;    // experts of the lane still to choose from
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t key = order_key(c[i]);
            key = key ? key : 1;
            if (((left >> i) & 1u) && key > best) {
                best = key;
                at = i;
            }
        }
        const uint64_t M = group_max64<L>(best);
        const int own = first_lane<L>(__ballot(best == M), seg);
        if (l == own) {
            left &= ~(1u << at);
            sel[j] = ex.first + at;
        }
    }
}

// Experts and weights of every token.
//
// s = softmax(x) or sigmoid(x); c = s (+ bias) chooses: with groups, a
// group's score is its largest c or the sum of its two largest, and the best
// `kept` groups stay; ids are the k largest c left, lowest index first among
// equals; w = s[ids], over their sum if renormalized, times scale.
//
// Bound by the vector ALU and by latency, not by memory: 16384 tokens of 256
// sigmoid scores in 8 groups take 12.0 us (919 vector instructions a wave, the
// ALU busy for 66% of it) where their bytes take 3.4 us; 128 softmax scores of one
// token 3.2 us, a launch's own time.
//
// L lanes hold one token, NV neighbouring experts each (64 / L tokens a
// wave), with the lanes of an expert group next to each other, so group
// scores and the k choices are reductions over lanes of one row of 16 where
// they fit (vector-ALU permutes, no LDS).  A choice keeps one number per
// lane, the largest key not yet taken: 28 bits of the ordered value and the
// place in the lane.  After a lane gives its head away, the next one is the
// largest key below it, max((key - head) mod 2^32), which needs no marking of
// taken experts.
//
// fp32 cannot order two scores that differ by less than its rounding.  The
// error of a score here is at most 4 half steps of fp32 for a sigmoid, 32 of
// the largest score for a softmax (half of it the sum's), and one for the
// bias; `margin` holds the double of the former, kRel that of the latter and
// of the 4 bits that a key drops.  Groups closer than that are scored again
// in fp64 (keep_fp64).  Where neighbours of the chosen order are, the list of
// choices is made a little longer, up to a clear gap, and sorted again by
// fp64 values, one expert a lane (no gap: choose_fp64).  About one wave in
// sixty takes these ways at 256 experts of fp32 logits and a random bias; the
// whole choice in fp64 in their place cost 10 us at 16384 tokens.  Equal scores
// (bf16 logits under equal biases) send most waves there: 16384 x 256 bf16 take
// 10.4 us with a zero bias, 9.2 with a random one (softmax 15.4 and 11.7; in 8
// groups with two scores each 13.3 and 10.7).  Without a bias the order of s is that
// of x: bf16 logits are then compared exactly (16 bits of value fit the key),
// fp32 ones sorted again by the logit itself.
template <int L, int NV, class E>
__global__ __launch_bounds__(kBlock, 4) void route_kernel(const RouteArgs a) {
    __shared__ int sel[kBlock / L][L];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int seg = lane & ~(L - 1), l = lane & (L - 1);
    const int slot = wave * (64 / L) + lane / L;
    const int64_t token = (int64_t)blockIdx.x * (kBlock / L) + slot;
    const bool live = token < a.T;
    const E *row = static_cast<const E *>(a.x) + (live ? token : a.T - 1) * a.ld;
    const LaneExperts ex = lane_experts<NV>(a, l);
    const float kNone = -__builtin_inff();

    float v[NV], bias[NV];
    load_values<NV>(row + (ex.count ? ex.first : 0), ex.count, kNone, v);
    if (a.bias) load_values<NV>(a.bias + (ex.count ? ex.first : 0), ex.count, 0.0f, bias);
    if (a.order_x) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += 0.0f;       // -0 as 0: equal logits get equal keys (scores are never -0)
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = __builtin_fmaxf(top, v[i]);
    top = group_reduce<L>(top, OpMax());

    // scores for the choice; the weights are computed again from the chosen
    // logits, at full accuracy
    float inv = 1.0f, margin = 0x1p-20f;
    if (a.sigmoid) {
        if (!a.order_x) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = fast_sigmoid(v[i]);
        }
    } else {
        float s[NV], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = __builtin_amdgcn_exp2f((v[i] - top) * kLog2E);
            sum += i < ex.count ? s[i] : 0.0f;
        }
        inv = 1.0f / group_reduce<L>(sum, OpAdd());
        margin = 0x1p-18f * inv;
        if (!a.order_x) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = s[i] * inv;
        }
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += bias[i];
    }

    const float kRel = 0x1p-18f;
    bool keep = ex.g < a.groups;
    if (a.groups > 1) {
        float b1 = kNone, b2 = kNone;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float y = i < ex.count ? v[i] : kNone;
            b2 = __builtin_fmaxf(b2, __builtin_fminf(b1, y));
            b1 = __builtin_fmaxf(b1, y);
        }
#pragma unroll
        for (int step = 0; step < 6; ++step) {
            if (step >= a.lanes_shift) break;
            float o1, o2;
            switch (step) {
                case 0: o1 = partner<0>(b1); o2 = partner<0>(b2); break;
                case 1: o1 = partner<1>(b1); o2 = partner<1>(b2); break;
                case 2: o1 = partner<2>(b1); o2 = partner<2>(b2); break;
                case 3: o1 = partner<3>(b1); o2 = partner<3>(b2); break;
                case 4: o1 = partner<4>(b1); o2 = partner<4>(b2); break;
                default: o1 = partner<5>(b1); o2 = partner<5>(b2); break;
            }
            b2 = __builtin_fmaxf(__builtin_fminf(b1, o1), __builtin_fmaxf(b2, o2));
            b1 = __builtin_fmaxf(b1, o1);
        }
        const float score = a.group_top == 2 ? b1 + b2 : b1;
        const uint32_t mine = order_key(score);
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint32_t o = (uint32_t)__shfl((int)mine, seg + (g << a.lanes_shift), 64);
            rank += (o > mine || (o == mine && g < ex.g)) ? 1 : 0;
        }
        const bool in = keep;
        keep = keep && rank < a.kept;
        if (!a.order_x) {
            // what a group's score may be off by goes by its terms, which can be far larger than their sum
            const float off = margin + kRel * (__builtin_fabsf(b1) + (a.group_top == 2 ? __builtin_fabsf(b2) : 0.0f));
            const float low = group_reduce<L>(keep ? score - off : __builtin_inff(), OpMin());
            const float high = group_reduce<L>(in && !keep ? score + off : kNone, OpMax());
            const bool close = !(low > high);
            if (__ballot(close && live)) {
                const float bar = a.group_top == 2 ? b2 : b1;
                keep = keep_fp64<L, NV, E>(a, row, ex, fp64_row<L, E>(a, row, ex, top), v,
                                           bar - (2.0f * margin + kRel * __builtin_fabsf(bar)), lane);
            }
        }
    }

    uint32_t key[NV];
    uint32_t head = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint32_t u = order_key(v[i]);
        u = u > 16u ? u : 16u;
        key[i] = (i < ex.count && keep) ? ((u & ~15u) | (uint32_t)(15 - i)) : 0u;
        head = key[i] > head ? key[i] : head;
    }
    uint32_t mine = 0;                             // lane j: the j-th largest key
    // choices j0 .. j1 - 1 of every token
    auto choose = [&](int j0, int j1) {
        for (int j = j0; j < j1; ++j) {
            const uint32_t hv = head & ~15u;
            const uint32_t M = group_reduce<L>(hv, OpMax());
            const int own = first_lane<L>(__ballot(hv == M), seg);
            if (l == j) mine = M;
            if (l == own) {
                sel[slot][j] = ex.first + 15 - (int)(head & 15u);
                uint32_t d = 0u - head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const uint32_t e = key[i] - head;
                    d = e > d ? e : d;
                }
                head += d;
            }
        }
        wave_sync();
    };
    // the logit of the listed expert of the lane, and whether its place before
    // the next lane's is beyond doubt
    int count = a.k + (a.order_exact || a.k == a.candidates ? 0 : 1);
    int id = 0;
    float x = 0.0f;
    auto listed = [&]() {
        id = l < count ? sel[slot][l] : 0;
        x = Elem<E>::get(row[id]);
        if (a.order_exact) return true;
        float c = x;
        if (!a.order_x) {
            c = a.sigmoid ? fast_sigmoid(x) : __builtin_amdgcn_exp2f((x - top) * kLog2E) * inv;
            if (a.bias) c += a.bias[id];
        }
        const uint32_t next = (uint32_t)__shfl_down((int)mine, 1, 64);
        const float below = __shfl_down(c, 1, 64);
        return mine != next && (a.order_x || c - below > margin + kRel * __builtin_fabsf(c));
    };
    choose(0, count);
    bool clear = listed();
    if (__ballot(!clear && l + 1 < count && live)) {
        const int more = a.candidates < L ? a.candidates : L;
        const int longer = count + 3 < more ? count + 3 : more;
        choose(count, longer);
        count = longer;
        clear = listed();
        // lanes of the token whose place ends a list that holds every contender for the k
        const uint64_t ends = __ballot(clear && l >= a.k - 1 && l + 1 < count);
        const bool whole = count == a.candidates || first_lane<L>(ends, seg) < L;
        const Fp64Row r = fp64_row<L, E>(a, row, ex, top);
        if (__ballot(!whole && live)) {
            wave_sync();
            choose_fp64<L, NV, E>(a, row, ex, r, keep, lane, sel[slot]);
        } else {
            uint64_t value = order_key(fp64_value(a, r, x, id));
            int rank = 0;
            for (int j = 0; j < count; ++j) {
                const uint64_t o = shfl64(value, seg + j);
                const int other = __shfl(id, seg + j, 64);
                rank += (o > value || (o == value && other < id)) ? 1 : 0;
            }
            wave_sync();
            if (l < count && rank < a.k) sel[slot][rank] = id;
        }
        wave_sync();
        id = l < a.k ? sel[slot][l] : 0;
        x = Elem<E>::get(row[id]);
    }

    float w = 0.0f;
    if (l < a.k) w = a.sigmoid ? sigmoid(x) : exp_neg(x - top) * inv;
    if (a.renorm) {
        float sum = group_reduce<L>(w, OpAdd());
        if (__ballot(sum < kSmallSum)) {
            const Shares r = shares<L>(x, l < a.k, a.sigmoid);
            w = sum < kSmallSum ? r.part : w;
            sum = sum < kSmallSum ? r.sum : sum;
        }
        w = w / sum;
    }
    if (live && l < a.k) {
        a.ids[token * a.k + l] = id;
        a.w[token * a.k + l] = w * a.scale;
    }
}

// Gradient of the weights with respect to the logits.
//
// With g = d_w * scale, a = s[ids], A = sum a: renormalized weights a / A give
// ds = (g - sum(g a) / A) / A on the chosen experts, else ds = g.  softmax:
// dx = s (ds - sum(ds a)) over all experts; sigmoid: dx = ds s (1 - s) on the
// chosen ones, 0 elsewhere.  One read of the logits (softmax) and one write;
// lanes as in route_kernel, the chosen experts' ds spread over the row
// through LDS.
template <int L, int NV, class E>
__global__ __launch_bounds__(kBlock) void route_backward_kernel(const RouteArgs a) {
    __shared__ float full[kBlock / L][L * NV];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = lane & (L - 1);
    const int slot = wave * (64 / L) + lane / L;
    const int64_t token = (int64_t)blockIdx.x * (kBlock / L) + slot;
    const bool live = token < a.T;
    const int64_t t = live ? token : a.T - 1;
    const E *row = static_cast<const E *>(a.x) + t * a.ld;
    const int first = l * NV;
    int count = a.E - first;
    count = count < 0 ? 0 : count > NV ? NV : count;

    float *mine = &full[slot][first];
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[i] = 0.0f;
    int id = -1;
    float g = 0.0f, x = 0.0f;
    if (l < a.k) {
        id = a.ids[t * a.k + l];
        g = a.dw[t * a.k + l] * a.scale;
        if (id < 0 || id >= a.E) id = -1;
        else x = Elem<E>::get(row[id]);
    }
    float s[NV], inv = 1.0f, top = 0.0f;
    if (!a.sigmoid) {
        float v[NV];
        load_values<NV>(row + (count ? first : 0), count, -__builtin_inff(), v);
        top = v[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) top = __builtin_fmaxf(top, v[i]);
        top = group_reduce<L>(top, OpMax());
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = i < count ? exp_neg(v[i] - top) : 0.0f;
            sum += s[i];
        }
        inv = 1.0f / group_reduce<L>(sum, OpAdd());
    }
    float chosen = 0.0f;
    if (id >= 0) chosen = a.sigmoid ? sigmoid(x) : exp_neg(x - top) * inv;
    else g = 0.0f;
    float ga = group_reduce<L>(g * chosen, OpAdd());
    float slope = chosen * (a.sigmoid ? sigmoid(-x) : 1.0f);         // ds / dx: 1 - s(x) = s(-x), without cancelling
    bool small = false;
    if (a.renorm) {
        const float A = group_reduce<L>(chosen, OpAdd());
        small = A < kSmallSum;
        float direct = 0.0f, mean = 0.0f;
        if (__ballot(small)) {                                       // dx = w (g - sum(g w)), times s(-x)
            const Shares r = shares<L>(x, id >= 0, a.sigmoid);
            const float w = id >= 0 ? r.part / r.sum : 0.0f;
            mean = group_reduce<L>(g * w, OpAdd());
            direct = w * (a.sigmoid ? sigmoid(-x) : 1.0f) * (g - mean);
        }
        g = (g - ga / A) / A;
        ga = group_reduce<L>(id >= 0 ? g * chosen : 0.0f, OpAdd());
        if (small) g = direct, slope = 1.0f, ga = mean - mean;
    }
    const bool whole = a.sigmoid || small;                           // the chosen experts' gradients are all there is
    wave_sync();
    if (id >= 0) full[slot][id] = whole ? g * slope : g;
    wave_sync();
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = a.sigmoid ? mine[i] : small ? mine[i] + ga : s[i] * inv * (mine[i] - ga);
    if (!live) return;
    E *out = static_cast<E *>(a.dx) + token * a.E + first;
    if constexpr (NV >= Elem<E>::kVec) {
        if (count == NV) {
#pragma unroll
            for (int i = 0; i < NV; i += Elem<E>::kVec) store16(out + i, Elem<E>::pack(d + i));
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < count) out[i] = Elem<E>::put(d[i]);
}

template <int L, int NV>
void start_route(const RouteArgs &a, bool bf16, bool backward, hipStream_t stream) {
    const unsigned grid = (unsigned)ceil_div(a.T, kBlock / L);
    if (backward) {
        if (bf16) route_backward_kernel<L, NV, uint16_t><<<grid, kBlock, 0, stream>>>(a);
        else route_backward_kernel<L, NV, float><<<grid, kBlock, 0, stream>>>(a);
    } else {
        if (bf16) route_kernel<L, NV, uint16_t><<<grid, kBlock, 0, stream>>>(a);
        else route_kernel<L, NV, float><<<grid, kBlock, 0, stream>>>(a);
    }
}

// Lanes per token L and experts per lane NV: as few lanes as hold the experts
// at 16 a lane (more tokens a wave, shorter reductions), at least 16 and more
// than k.
hipError_t start(RouteArgs a, bool bf16, bool backward, hipStream_t stream) {
    int groups2 = 1, gshift = 0;
    while (groups2 < a.groups) groups2 <<= 1, ++gshift;
    int shift = 4;
    int64_t nv = 0;
    for (;; ++shift) {
        if ((1 << shift) <= a.k || shift < gshift) continue;
        a.lanes_shift = shift - gshift;
        nv = ceil_div(a.size, (int64_t)1 << a.lanes_shift);
        if (nv <= 16) break;
        if (shift == 6) return hipErrorInvalidValue;
    }
    if (shift == 4) {
        if (nv == 1) start_route<16, 1>(a, bf16, backward, stream);
        else if (nv == 2) start_route<16, 2>(a, bf16, backward, stream);
        else if (nv <= 4) start_route<16, 4>(a, bf16, backward, stream);
        else if (nv <= 8) start_route<16, 8>(a, bf16, backward, stream);
        else start_route<16, 16>(a, bf16, backward, stream);
    } else if (shift == 5) {
        if (nv <= 8) start_route<32, 8>(a, bf16, backward, stream);
        else start_route<32, 16>(a, bf16, backward, stream);
    } else {
        if (nv <= 8) start_route<64, 8>(a, bf16, backward, stream);
        else start_route<64, 16>(a, bf16, backward, stream);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, bool bf16, hipStream_t stream) {
    RouteArgs a = args;
    if (a.kept == a.groups) {                        // every group stays: one group
        a.groups = a.kept = 1;
        a.size = a.E;
    }
    // without a bias s rises with x, so the choice (and a group's largest) can be read off x
    a.order_x = !a.bias && (a.groups == 1 || a.group_top == 1);
    a.order_exact = a.order_x && bf16;
    a.candidates = a.kept * a.size;
    return start(a, bf16, false, stream);
}

hipError_t launch_route_backward(const RouteArgs &args, bool bf16, hipStream_t stream) {
    RouteArgs a = args;
    a.groups = a.kept = 1;
    a.size = a.E;
    return start(a, bf16, true, stream);
}

}  // namespace mx
