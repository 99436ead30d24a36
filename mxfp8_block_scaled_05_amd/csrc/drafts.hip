// Which drafted tokens stand against the target's probabilities, and the token
// that follows them.
//
//   rows    max and sum of e^((x - max) / temp) of every row of the target's
//           and the draft's logits: one pass over all of them
//   draw    where each request stops, and the race of w / noise at that row,
//           split over blocks
//   finish  joins the race and writes the token (by the last block of a race
//           instead: 64 requests 106 us for 50, since the fences that it needs
//           write back and empty each XCD's L2)
//
// Whether a token stands, and which column wins, are decisions of whole
// numbers that a last bit can turn.  They are taken from fp32 exponentials
// with a bound of what those may be off by; where the bound leaves two
// outcomes, the decision is taken again in fp64, by one block over whole rows:
// a request of a batch of 64 that needs it takes the call from 45 us to 435.
// How often: whether a token stands, and a race of p alone, about 1 time in
// 10^4.  A race of p - q is bounded by 2^-15 (p + q), so it is open the more
// often the less p and q differ, but then fewer tokens are refused at all: of
// 15360 tokens over 131072 columns, drafted from logits off by 0.7 (0.1, 0.02,
// 0.005), 4404 (640, 156, 41) were refused and 1 (0, 2, 2) races open.
//
// Bounds.  A term's exponent carries three roundings of |u| 2^-24 (distance,
// scale, product), u its distance from the maximum in powers of two.  Averaged
// over a row |u| is at most log2 V, so the terms of a row's sum, whose groups of
// 32 are added in fp64, are off by 31 * 3 * ln 2 * 2^-24 + 2^-21 < 2^-17.8 of it.
// Where a maximum rises, the sum so far is scaled by an exponential that is off
// by 2^-23 at most, whatever the rise (the errors of rises too small for it all
// have one sign).  A slice of kSlice columns has 64 groups of 4096 fp32 columns
// at most, 4 at its end and 2 joins, 70 * 2^-23 < 2^-16.8; slices are joined in
// fp64.  Together a row's sum is within 2^-16.2 of its value.  A single term of
// |u| <= 126 is within 126 * 3 * ln 2 * 2^-24 + 2^-22 < 2^-15.9; below it is 0.
#include <type_traits>

#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;
constexpr int kUnroll = 4;
constexpr int kDrawBlocks = 4;              // of the race resident on a compute unit
constexpr float kLowest = -3.402823466e38f;
constexpr int64_t kSlice = 1 << 18;         // columns of a slice at most
constexpr float kDrawSlack = 0x1p-15f;      // of p and q as the race sees them: a term and the row's sum
constexpr double kStandSlack = 0x1p-16;     // of p(x) and u q(x): their terms in fp64, the rows' sums as above

// A row's largest logit and the sum of e^((x - m) / temp).
struct RowSum {
    float m;
    double s;
};
struct Pair {
    RowSum p, q;
};
struct Part {                               // of a slice of a row, in the workspace
    float m, pad;
    double s;
};
__device__ __forceinline__ Part *parts_of(const DraftArgs &a) { return static_cast<Part *>(a.workspace); }

// The best of a race: the largest upper bound of w / noise and its column
// (-1: no w above 0), and the next largest.
struct Race {
    float best, second;
    int column;
};
// What the fast sums say about a request, from its first draw block to finish.
struct Verdict {
    int end;                                // drafted tokens that stand
    int open;                               // finish takes the decisions and writes the tokens
    Pair rows;                              // at which it stops
};
__device__ __forceinline__ Verdict *verdicts_of(const DraftArgs &a) {
    return reinterpret_cast<Verdict *>(parts_of(a) + a.rows * a.slices);
}
__device__ __forceinline__ Race *races_of(const DraftArgs &a) { return reinterpret_cast<Race *>(verdicts_of(a) + a.B); }

template <int W>
__device__ __forceinline__ double sum_lanes(double v) {
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// N logits of every lane into its running maximum and sum; one new maximum and
// one rescaling for them together
template <int N>
__device__ __forceinline__ void take(RowSum &v, const float *x, float c) {
    float g = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) g = __builtin_fmaxf(g, x[i]);
    const float m = __builtin_fmaxf(v.m, g);
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = __builtin_amdgcn_exp2f((x[i] - m) * c);
#pragma unroll
    for (int n = N / 2; n; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) e[i] += e[i + n];
    v.s = v.s * (double)__builtin_amdgcn_exp2f((v.m - m) * c) + (double)e[0];
    v.m = m;
}

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

// Row i of the target (i < R) or row i - R of the draft
template <class E>
__device__ __forceinline__ const E *row_of(const DraftArgs &a, int64_t i) {
    return i < a.R ? static_cast<const E *>(a.x) + i * a.ld : static_cast<const E *>(a.d) + (i - a.R) * a.ld_d;
}

// One pass, bound by HBM where there are many: 512 rows of 131072 bf16 (134 MB)
// 22.7 us, 5.9 TB/s with the vector ALU at 66%; 198 rows of 100003 fp32 15 us, 5.3.
template <class E, int BLOCK, bool ONCE>
__global__ __launch_bounds__(BLOCK) void draft_rows_kernel(const DraftArgs a) {
    constexpr int kV = Elem<E>::kVec, kWaves = BLOCK / 64, kStep = BLOCK * kV;
    __shared__ Part parts[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x / a.slices;
    const int slice = (int)((int64_t)blockIdx.x - t * a.slices);
    const int64_t lo = slice * a.slice;
    const int64_t hi = lo + a.slice < a.V ? lo + a.slice : a.V;
    const E *row = row_of<E>(a, t);
    const float c = a.scale;
    RowSum v{kLowest, 0.0};
    int64_t col = lo + threadIdx.x * kV, base = lo;
    for (; base + kUnroll * kStep <= hi; base += kUnroll * kStep, col += kUnroll * kStep) {
        v4u r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) r[u] = load16<ONCE>(row + col + u * kStep);
        float x[kUnroll * kV];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) Elem<E>::unpack(r[u], x + u * kV);
        take<kUnroll * kV>(v, x, c);
    }
    for (; base < hi; base += kStep, col += kStep) {
        float x[kV];
        load_logits(row + col, hi - col, x);
        take<kV>(v, x, c);
    }
    const float m = group_reduce<64>(v.m, OpMax());
    const double s = sum_lanes<64>(v.s * (double)__builtin_amdgcn_exp2f((v.m - m) * c));
    if (lane == 0) parts[wave] = Part{m, 0.0f, s};
    __syncthreads();
    if (threadIdx.x != 0) return;
    Part p = parts[0];
    for (int i = 1; i < kWaves; ++i) p.m = __builtin_fmaxf(p.m, parts[i].m);
    p.s = 0.0;
    for (int i = 0; i < kWaves; ++i) p.s += parts[i].s * (double)__builtin_amdgcn_exp2f((parts[i].m - p.m) * c);
    parts_of(a)[blockIdx.x] = p;
}

// The joined slices of two rows (the second may be none, -1: sum 1), half a
// wave each; all lanes get both.  A row with a NaN or +Inf, or nothing above
// -Inf, has s = NaN.
__device__ __forceinline__ Pair join_rows(const DraftArgs &a, int64_t i, int64_t j, int lane) {
    const int64_t row = lane < 32 || j < 0 ? i : j;
    const Part *part = parts_of(a) + row * a.slices;
    const int l = lane & 31;
    Part held = part[l < a.slices ? l : 0];              // at most 32 of them as a rule
    if (l >= a.slices) held.s = 0.0;
    float m = held.m;
    for (int k = l + 32; k < a.slices; k += 32) m = __builtin_fmaxf(m, part[k].m);
    m = group_reduce<32>(m, OpMax());
    double s = held.s * exp2(((double)held.m - m) * a.scale64);
    for (int k = l + 32; k < a.slices; k += 32) s += part[k].s * exp2(((double)part[k].m - m) * a.scale64);
    s = sum_lanes<32>(s);
    if (!(s > 0.0) || m > -kLowest) s = __builtin_nan("");
    Pair r{{__shfl(m, 0, 64), __shfl(s, 0, 64)}, {__shfl(m, 32, 64), __shfl(s, 32, 64)}};
    if (j < 0) r.q = RowSum{0.0f, 1.0};
    return r;
}

// p or q of a logit of a row, in fp64 but for the row's sum
__device__ __forceinline__ double share(const DraftArgs &a, double x, const RowSum &r) {
    return exp2((x - r.m) * a.scale64) / r.s;
}

// The rows of a request: `drafts` drafted ones from row `first` on and one
// more (drafts < 0: none at all); their drafted tokens from `draft` on.
struct Request {
    int64_t first, draft;
    int drafts;
};
__device__ __forceinline__ Request request_of(const DraftArgs &a, int64_t b) {
    int64_t lo = a.offsets[b], hi = a.offsets[b + 1];
    lo = lo < 0 ? 0 : lo > a.R ? a.R : lo;
    hi = hi < lo ? lo : hi > a.R ? a.R : hi;
    const int64_t draft = lo - b, most = a.R - a.B - draft;
    int64_t n = hi - lo - 1;
    if (n > 0 && (draft < 0 || n > most)) n = draft < 0 || most < 0 ? 0 : most;     // a malformed table
    return {lo, draft, (int)n};
}

// Whether drafted token i of a request stands; close: fp64 sums might say
// otherwise.
struct Stand {
    bool stands, close;
    int64_t id;
    float logprob;
};
__device__ __forceinline__ float log_share(const DraftArgs &a, double x, const RowSum &r) {
    return (float)((x - r.m) * a.inv_temperature - log(r.s));
}
template <class E>
__device__ __forceinline__ Stand stand_of(const DraftArgs &a, const Request &r, int i, int64_t x, double u, const Pair &rows) {
    if (x < 0 || x >= a.V) return {false, false, x, 0.0f};
    const double z = Elem<E>::get(row_of<E>(a, r.first + i)[x]);
    const double p = share(a, z, rows.p);
    const double q = a.d ? share(a, Elem<E>::get(row_of<E>(a, a.R + r.draft + i)[x]), rows.q) : 1.0;
    const double uq = u * q;
    return {uq < p, uq + p > 0.0 && __builtin_fabs(uq - p) <= kStandSlack * (uq + p), x, log_share(a, z, rows.p)};
}
// that of the rows' fast sums; all lanes of a wave
template <class E>
__device__ __forceinline__ Stand fast_stand(const DraftArgs &a, const Request &r, int i, int lane, Pair &rows) {
    const int64_t x = a.ids[r.draft + i];
    const float u = a.u[r.draft + i];
    rows = join_rows(a, r.first + i, a.d ? a.R + r.draft + i : -1, lane);
    return stand_of<E>(a, r, i, x, u, rows);
}

// Where a request of at most kHeld drafted tokens stops by the fast sums, with
// the sums of all its rows.  In LDS, by the whole block.  Requests of more are
// left to the fp64 race: one of 31 drafted tokens over 131072 columns takes 30 us,
// one of 32 to 40 288 us, eight of 40 314.
constexpr int kHeld = 31;
struct Held {
    int refused, close;             // the first of each
    Pair rows[kHeld + 1];
    Stand stand[kHeld + 1];
};
template <class E>
__device__ __forceinline__ void hold(const DraftArgs &a, const Request &r, Held &h) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) h.refused = h.close = r.drafts;
    __syncthreads();
    for (int i = wave; i <= r.drafts; i += kBlock / 64) {
        Pair rows;
        Stand s{true, false, -1, 0.0f};
        if (i < r.drafts) s = fast_stand<E>(a, r, i, lane, rows);
        else rows = join_rows(a, r.first + i, -1, lane);
        if (lane == 0) {
            h.rows[i] = rows, h.stand[i] = s;
            if (!s.stands) atomicMin(&h.refused, i);
            if (s.close) atomicMin(&h.close, i);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void merge(Race &v, const Race &o) {
    const bool first = o.best > v.best || (o.best == v.best && o.column >= 0 && (v.column < 0 || o.column < v.column));
    const float low = first ? v.best : o.best;
    v.second = __builtin_fmaxf(__builtin_fmaxf(v.second, o.second), low);
    if (first) v.best = o.best, v.column = o.column;
}
__device__ __forceinline__ Race merge_lanes(Race v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        merge(v, Race{__shfl_xor(v.best, d, 64), __shfl_xor(v.second, d, 64), __shfl_xor(v.column, d, 64)});
    return v;
}

// ---------------------------------------------------------------- draw

// A cut of the race at the row where a request stops.  Every column's upper
// bound of w / noise, with w = p - q; the column that wins does so for certain
// if its lower bound is above the next upper bound.  A request's first block
// writes the drafted tokens that stand and what is behind the next one.  Bound by
// the exponentials of both distributions and their bounds (vector ALU 67%): 64
// requests of 131072 columns 17 us, 33 of 100003 without a draft 12.
template <class E>
__global__ __launch_bounds__(kBlock, kDrawBlocks) void draft_draw_kernel(const DraftArgs a) {
    constexpr int kV = Elem<E>::kVec, kStep = kBlock * kV;
    __shared__ Held held;
    __shared__ Race races[kBlock / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x / a.cuts;
    const int cut = (int)(blockIdx.x - b * a.cuts);
    const Request r = request_of(a, b);
    if (r.drafts < 0) return;
    Verdict &verdict = verdicts_of(a)[b];
    bool open = r.drafts > kHeld;
    if (!open) {
        hold<E>(a, r, held);
        open = held.close <= held.refused && held.close < r.drafts;
    }
    if (cut == 0 && threadIdx.x == 0) {
        verdict.end = open ? 0 : held.refused, verdict.open = open;
        if (!open) verdict.rows = held.rows[held.refused];
    }
    if (open) return;
    const int end = held.refused;
    if (cut == 0 && threadIdx.x <= r.drafts && threadIdx.x != end) {
        const Stand s = held.stand[threadIdx.x];
        const bool stands = (int)threadIdx.x < end;
        a.tokens[r.first + threadIdx.x] = stands ? s.id : -1;
        a.logprobs[r.first + threadIdx.x] = stands ? s.logprob : 0.0f;
    }
    const int64_t at = r.first + end, drafted = r.draft + end;
    const bool refused = end < r.drafts, with_q = refused && a.d;
    const Pair rows = held.rows[end];
    const int64_t named = held.stand[end].id;
    const int taken = refused && !a.d && named >= 0 && named < a.V ? (int)named : -1;
    const float pk = (float)((1.0 + kDrawSlack) / rows.p.s), qk = with_q ? (float)((1.0 - kDrawSlack) / rows.q.s) : 0.0f;
    const E *x = row_of<E>(a, at), *d = with_q ? row_of<E>(a, a.R + drafted) : x;
    const float *noise = a.noise + b * a.ld_n;
    const float c = a.scale, pm = rows.p.m, qm = with_q ? rows.q.m : rows.p.m;
    const int64_t lo64 = cut * a.cut, hi64 = lo64 + a.cut < a.V ? lo64 + a.cut : a.V;
    const int lo = (int)lo64, hi = (int)hi64, off = threadIdx.x * kV;            // V < 2^31
    Race v{0.0f, 0.0f, -1};
    auto race = [&](auto two) {
        constexpr bool kTwo = decltype(two)::value;      // w = p - q
        auto offer = [&](const float *xs, const float *ds, const float *ns, int col) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float w = __builtin_amdgcn_exp2f((xs[i] - pm) * c) * pk;
                if constexpr (kTwo) w = __builtin_fmaxf(w - __builtin_amdgcn_exp2f((ds[i] - qm) * c) * qk, 0.0f);
                float t = w * __builtin_amdgcn_rcpf(ns[i]);
                if constexpr (!kTwo) t = col + i == taken ? 0.0f : t;
                const bool first = t > v.best;
                v.second = __builtin_fmaxf(v.second, first ? v.best : t);
                v.best = first ? t : v.best;
                v.column = first ? col + i : v.column;
            }
        };
        int base = lo;
        auto steps = [&](auto ahead) {                   // that many loads of each kind in flight
            constexpr int kAhead = decltype(ahead)::value;
            for (; hi - base >= kAhead * kStep; base += kAhead * kStep) {
                const int col = base + off;
                v4u xr[kAhead], dr[kAhead], nr[kAhead][kV / 4];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    xr[u] = load16(x + col + u * kStep);
                    if constexpr (kTwo) dr[u] = load16(d + col + u * kStep);
#pragma unroll
                    for (int i = 0; i < kV; i += 4) nr[u][i / 4] = load16(noise + col + u * kStep + i);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float xs[kV], ds[kV], ns[kV];
                    Elem<E>::unpack(xr[u], xs);
                    if constexpr (kTwo) Elem<E>::unpack(dr[u], ds);
#pragma unroll
                    for (int i = 0; i < kV; i += 4) Elem<float>::unpack(nr[u][i / 4], ns + i);
                    offer(xs, ds, ns, col + u * kStep);
                }
            }
        };
        steps(std::integral_constant<int, 2>());
        steps(std::integral_constant<int, 1>());
        if (hi - base > off) {                           // less than a step is left
            float xs[kV], ds[kV], ns[kV];
            const int col = base + off, n = hi - col;
            load_logits(x + col, n, xs);
            if constexpr (kTwo) load_logits(d + col, n, ds);
            if (n >= kV) {
#pragma unroll
                for (int i = 0; i < kV; i += 4) Elem<float>::unpack(load16(noise + col + i), ns + i);
            } else {
                load_head<kV>(noise + col, n, 1.0f, ns);
            }
            offer(xs, ds, ns, col);
        }
    };
    if (with_q) race(std::true_type());
    else race(std::false_type());
    v = merge_lanes(v);
    if (lane == 0) races[wave] = v;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < kBlock / 64; ++i) merge(v, races[i]);
    races_of(a)[blockIdx.x] = v;
}

// ---------------------------------------------------------------- fp64

constexpr int kWide = 1024;         // threads of finish
constexpr int kWaves = kWide / 64;

__device__ __forceinline__ double sum_block(double v, double (&room)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = sum_lanes<64>(v);
    if (lane == 0) room[wave] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kWaves; ++i) v += room[i];
    __syncthreads();
    return v;
}

// kBatch values of a row in flight for a thread
constexpr int kBatch = 8;
template <class E>
__device__ __forceinline__ void load_batch(const E *x, int64_t col0, int64_t V, float (&v)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t col = col0 + k * kWide;
        v[k] = Elem<E>::get(x[col < V ? col : 0]);
    }
}

// A row's sum in fp64 over the same maximum
template <class E>
__device__ __forceinline__ RowSum exact_row(const DraftArgs &a, int64_t i, const RowSum &fast, double (&room)[kWaves]) {
    const E *x = row_of<E>(a, i);
    double s = 0.0;
    for (int64_t col0 = threadIdx.x; col0 < a.V; col0 += kWide * kBatch) {
        float v[kBatch];
        load_batch(x, col0, a.V, v);
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k)
            if (col0 + k * kWide < a.V) s += exp2(((double)v[k] - fast.m) * a.scale64);
    }
    s = sum_block(s, room);
    return {fast.m, fast.s == fast.s ? s : fast.s};
}

struct Exact {
    double score;
    int64_t column;
};
__device__ __forceinline__ void better(Exact &v, const Exact &o) {
    if (o.column >= 0 && (v.column < 0 || o.score > v.score || (o.score == v.score && o.column < v.column))) v = o;
}

// The race in fp64: w = p - q, or p without q (`taken`: that column is left out)
template <class E>
__device__ __forceinline__ int64_t exact_race(const DraftArgs &a, int64_t b, int64_t at, const RowSum &pr, int64_t q_at,
                                              const RowSum &qr, int64_t taken, Exact (&room)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const E *x = row_of<E>(a, at), *d = q_at < 0 ? x : row_of<E>(a, q_at);
    Exact v{0.0, -1};
    for (int64_t col0 = threadIdx.x; col0 < a.V; col0 += kWide * kBatch) {
        float xs[kBatch], ds[kBatch], ns[kBatch];
        load_batch(x, col0, a.V, xs);
        load_batch(d, col0, a.V, ds);
        load_batch(a.noise + b * a.ld_n, col0, a.V, ns);
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
            const int64_t col = col0 + k * kWide;
            double w = share(a, xs[k], pr);
            if (q_at >= 0) w -= share(a, ds[k], qr);
            const double score = w / (double)ns[k];
            if (w > 0.0 && score > 0.0 && col != taken && col < a.V) better(v, Exact{score, col});
        }
    }
#pragma unroll
    for (int n = 1; n < 64; n <<= 1) better(v, Exact{__shfl_xor(v.score, n, 64), __shfl_xor(v.column, n, 64)});
    if (lane == 0) room[wave] = v;
    __syncthreads();
    v = room[0];
    for (int i = 1; i < kWaves; ++i) better(v, room[i]);
    __syncthreads();
    return v.column;
}

// The token after the drafted ones, in fp64: of p - q (q_at < 0: of p without
// the column `taken`), or of p where that is nowhere above 0.
template <class E>
__device__ __forceinline__ int64_t exact_draw(const DraftArgs &a, int64_t b, int64_t at, const Pair &fast, int64_t q_at, bool refused,
                                              int64_t taken, double (&sums)[kWaves], Exact (&exacts)[kWaves]) {
    if (fast.p.s != fast.p.s) return -1;                 // a row without a distribution
    const RowSum p = exact_row<E>(a, at, fast.p, sums);
    RowSum q = fast.q;
    if (q_at >= 0) q = exact_row<E>(a, q_at, q, sums);
    int64_t token = exact_race<E>(a, b, at, p, q_at, q, taken, exacts);
    if (token < 0 && refused) token = exact_race<E>(a, b, at, p, -1, q, -1, exacts);
    return token;
}

template <class E>
__device__ __forceinline__ void put_token(const DraftArgs &a, int64_t b, int64_t at, int end, int64_t token, const RowSum &p) {
    a.accepted[b] = end;
    a.tokens[at] = token;
    a.logprobs[at] = token >= 0 ? log_share(a, Elem<E>::get(row_of<E>(a, at)[token]), p) : __builtin_nanf("");
}

// A request whose decisions the fast sums leave open, or with more drafted
// tokens than are held: one after another, the close ones in fp64, and the race
// in fp64.
template <class E>
__device__ __forceinline__ void resolve(const DraftArgs &a, const Request &r, int64_t b, double (&sums)[kWaves], Exact (&exacts)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int end = 0;
    for (; end < r.drafts; ++end) {
        Pair rows;
        Stand s = fast_stand<E>(a, r, end, lane, rows);
        if (s.close) {
            rows.p = exact_row<E>(a, r.first + end, rows.p, sums);
            if (a.d) rows.q = exact_row<E>(a, a.R + r.draft + end, rows.q, sums);
            s = stand_of<E>(a, r, end, s.id, a.u[r.draft + end], rows);
        }
        if (!s.stands) break;
    }
    const bool refused = end < r.drafts;
    const int64_t q_at = refused && a.d ? a.R + r.draft + end : -1;
    const Pair rows = join_rows(a, r.first + end, q_at, lane);
    const int64_t token = exact_draw<E>(a, b, r.first + end, rows, q_at, refused, refused && !a.d ? a.ids[r.draft + end] : -1, sums, exacts);
    if (threadIdx.x == 0) put_token<E>(a, b, r.first + end, end, token, rows.p);
    for (int i = wave; i <= r.drafts; i += kWaves) {
        if (i == end) continue;
        int64_t id = -1;
        float logprob = 0.0f;
        if (i < end) {
            Pair at;
            const Stand s = fast_stand<E>(a, r, i, lane, at);
            id = s.id, logprob = s.logprob;
        }
        if (lane == 0) a.tokens[r.first + i] = id, a.logprobs[r.first + i] = logprob;
    }
}

// One block a request; all of its waves take the same decisions.  A chain of
// latencies, 4.6 us for one request, 5.5 for 64.
template <class E>
__global__ __launch_bounds__(kWide) void draft_finish_kernel(const DraftArgs a) {
    __shared__ double sums[kWaves];
    __shared__ Exact exacts[kWaves];
    const int lane = threadIdx.x & 63;
    const int64_t b = blockIdx.x;
    const Request r = request_of(a, b);
    if (r.drafts < 0) {
        if (threadIdx.x == 0) a.accepted[b] = 0;
        return;
    }
    const Verdict verdict = verdicts_of(a)[b];
    Race v{0.0f, 0.0f, -1};
    for (int i = lane; i < a.cuts; i += 64) merge(v, races_of(a)[b * a.cuts + i]);
    if (verdict.open) {
        resolve<E>(a, r, b, sums, exacts);
        return;
    }
    v = merge_lanes(v);
    const Pair &rows = verdict.rows;
    const int64_t at = r.first + verdict.end, drafted = r.draft + verdict.end;
    const bool refused = verdict.end < r.drafts;
    const int64_t q_at = refused && a.d ? a.R + drafted : -1;
    int64_t token = -1;
    bool certain = !(rows.p.s == rows.p.s);              // a row without a distribution has no token
    if (!certain && v.column >= 0) {
        const double p = share(a, Elem<E>::get(row_of<E>(a, at)[v.column]), rows.p);
        const double q = q_at >= 0 ? share(a, Elem<E>::get(row_of<E>(a, q_at)[v.column]), rows.q) : 0.0;
        const double lower = ((1.0 - kDrawSlack) * p - (1.0 + kDrawSlack) * q) / (double)a.noise[b * a.ld_n + v.column];
        certain = (double)v.second < lower;
        token = v.column;
    }
    if (!certain) token = exact_draw<E>(a, b, at, rows, q_at, refused, refused && !a.d ? a.ids[drafted] : -1, sums, exacts);
    if (threadIdx.x == 0) put_token<E>(a, b, at, verdict.end, token, rows.p);
}

template <class E, bool ONCE>
void start_rows(const DraftArgs &a, int cus, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.rows * a.slices);
    // Many short rows: a wave each, without a join in LDS (all launches of 4000 rows of 1024 bf16 logits 30.8 us for 34.5,
    // 2000 of 4096 27.3 for 28.0; of 8192 fp32 42.5 for 41.5).
    if (a.rows >= 4 * cus && a.slice <= 4096) draft_rows_kernel<E, 64, ONCE><<<grid, 64, 0, stream>>>(a);
    else draft_rows_kernel<E, kBlock, ONCE><<<grid, kBlock, 0, stream>>>(a);
}
template <class E>
void start(const DraftArgs &a, int cus, hipStream_t stream) {
    // Past the caches where the logits are more than 3/8 of the last level, although the draws read some rows again:
    // 134 MB of bf16 logits 48.0 -> 45.3 us in all, 81 MB of fp32 logits 32.3 -> 32.6.
    if (a.rows * a.V * (int64_t)sizeof(E) > kLastLevelBytes / 8 * 3) start_rows<E, true>(a, cus, stream);
    else start_rows<E, false>(a, cus, stream);
    draft_draw_kernel<E><<<(unsigned)(a.B * a.cuts), kBlock, 0, stream>>>(a);
    draft_finish_kernel<E><<<(unsigned)a.B, kWide, 0, stream>>>(a);
}

}  // namespace

DraftCut draft_cut(int64_t rows, int64_t B, int64_t V, int cus) {
    // slices of a row: as few as kSlice allows where the rows alone give every compute unit a block, else enough for four
    // blocks each.  512 rows of 131072 bf16 logits 44.8 us, 45.2 to 45.7 in more slices.  Between the two sides some units
    // have two rows and most one: 504 rows 44.2 for 45.0 in two slices, 396 rows 42.2 for 41.3, 288 rows 37.3 for 33.5
    // (252 rows, four slices, 30.7); 258 rows of 100003 fp32 ones 43.0 for 38.1.
    int64_t slices = ceil_div(V, kSlice);
    if (rows < cus) {
        const int64_t want = ceil_div((int64_t)cus * 4, rows), most = ceil_div(V, 4096);
        const int64_t few = want < most ? want : most;
        slices = few > slices ? few : slices;
    }
    // cuts of a race: as many blocks as are resident at once, of at least 2048 columns
    const int64_t want = B < kDrawBlocks * (int64_t)cus ? kDrawBlocks * (int64_t)cus / B : 1, most = ceil_div(V, 2048);
    const int64_t cuts = want < most ? want : most;
    return {(int)slices, (int)cuts, ceil_div(ceil_div(V, slices), 8) * 8, ceil_div(ceil_div(V, cuts), 8) * 8,
            rows * slices * (int64_t)sizeof(Part) + B * ((int64_t)sizeof(Verdict) + cuts * (int64_t)sizeof(Race))};
}

hipError_t launch_drafts(DraftArgs a, bool bf16, hipStream_t stream) {
    const int cus = device_cu_count();
    const DraftCut cut = draft_cut(a.rows, a.B, a.V, cus);
    a.slices = cut.slices, a.cuts = cut.cuts, a.slice = cut.slice, a.cut = cut.cut;
    a.inv_temperature = 1.0 / a.temperature;
    a.scale64 = 1.4426950408889634 * a.inv_temperature;
    a.scale = (float)a.scale64;
    if (bf16) start<uint16_t>(a, cus, stream);
    else start<float>(a, cus, stream);
    return hipGetLastError();
}

}  // namespace mx
