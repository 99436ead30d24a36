// Which drafted tokens stand against the target's probabilities, and the token
// that follows them.
//
//   rows    max and sum of e^((x - max) / temp) of every row of the target's
//           and the draft's logits: one pass over all of them
//   draw    of the row at which each request stops: the race of w / noise,
//           split over blocks
//   finish  joins the race, writes the tokens and their log-probabilities
//
// Whether a token stands, and which column wins, are decisions of whole
// numbers that a last bit can turn.  They are taken from fp32 exponentials
// with a bound of what those may be off by; where the bound leaves two
// outcomes (about 1 request in 10^4), finish takes the decision again in fp64.
//
// Bounds.  A term's exponent carries three roundings of |u| 2^-24 (distance,
// scale, product), u its distance from the maximum in powers of two.  Averaged
// over a row |u| is at most log2 V, so a row's sum, whose groups of 32 terms
// are added in fp64, is within 31 * 3 * ln 2 * 2^-24 + 2^-21 < 2^-17 of its
// value (2^-18 at 2^17 columns).  A single term of |u| <= 126 is within
// 126 * 3 * ln 2 * 2^-24 + 2^-22 < 2^-15.9; below it is 0.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;
constexpr int kUnroll = 4;
constexpr float kLowest = -3.402823466e38f;
constexpr float kDrawSlack = 0x1p-15f;      // of p and q as the race sees them
constexpr double kStandSlack = 0x1p-16;     // of p(x) and u q(x): their terms in fp64, the rows' sums as above

// A row's largest logit and the sum of e^((x - m) / temp).
struct RowSum {
    float m;
    double s;
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
    int64_t column;
};
__device__ __forceinline__ Race *races_of(const DraftArgs &a) {
    return reinterpret_cast<Race *>(parts_of(a) + a.rows * a.slices);
}

__device__ __forceinline__ double sum_lanes(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
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
    const double s = sum_lanes(v.s * (double)__builtin_amdgcn_exp2f((v.m - m) * c));
    if (lane == 0) parts[wave] = Part{m, 0.0f, s};
    __syncthreads();
    if (threadIdx.x != 0) return;
    Part p = parts[0];
    for (int i = 1; i < kWaves; ++i) p.m = __builtin_fmaxf(p.m, parts[i].m);
    p.s = 0.0;
    for (int i = 0; i < kWaves; ++i) p.s += parts[i].s * (double)__builtin_amdgcn_exp2f((parts[i].m - p.m) * c);
    parts_of(a)[blockIdx.x] = p;
}

// The joined slices of row i; all lanes of a wave, all get it.  A row with a
// NaN or +Inf, or nothing above -Inf, has s = NaN.
__device__ __forceinline__ RowSum join_row(const DraftArgs &a, int64_t i, int lane) {
    const Part *p = parts_of(a) + i * a.slices;
    float m = kLowest;
    for (int k = lane; k < a.slices; k += 64) m = __builtin_fmaxf(m, p[k].m);
    m = group_reduce<64>(m, OpMax());
    double s = 0.0;
    for (int k = lane; k < a.slices; k += 64) s += p[k].s * exp2(((double)p[k].m - m) * a.scale64);
    s = sum_lanes(s);
    if (!(s > 0.0) || m > -kLowest) s = __builtin_nan("");
    return {m, s};
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
// otherwise.  All lanes of a wave.
struct Stand {
    bool stands, close;
};
template <class E>
__device__ __forceinline__ Stand stand_of(const DraftArgs &a, const Request &r, int i, const RowSum &p_row, const RowSum &q_row) {
    const int64_t x = a.ids[r.draft + i];
    if (x < 0 || x >= a.V) return {false, false};
    const double p = share(a, Elem<E>::get(row_of<E>(a, r.first + i)[x]), p_row);
    const double q = a.d ? share(a, Elem<E>::get(row_of<E>(a, a.R + r.draft + i)[x]), q_row) : 1.0;
    const double uq = (double)a.u[r.draft + i] * q;
    return {uq < p, uq + p > 0.0 && __builtin_fabs(uq - p) <= kStandSlack * (uq + p)};
}

// Where each request stops by the fast sums.  The whole block; `found` is LDS.
// end: the first drafted token that does not stand, or their number; close:
// a decision up to there needs fp64.
struct Stop {
    int end;
    bool close;
};
template <class E, int BLOCK>
__device__ __forceinline__ Stop stop_of(const DraftArgs &a, const Request &r, int (&found)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x < 2) found[threadIdx.x] = r.drafts < 0 ? 0 : r.drafts;
    __syncthreads();
    for (int i = wave; i < r.drafts; i += BLOCK / 64) {
        const RowSum p = join_row(a, r.first + i, lane);
        RowSum q{0.0f, 1.0};
        if (a.d) q = join_row(a, a.R + r.draft + i, lane);
        const Stand s = stand_of<E>(a, r, i, p, q);
        if (lane == 0 && !s.stands) atomicMin(&found[0], i);
        if (lane == 0 && s.close) atomicMin(&found[1], i);
    }
    __syncthreads();
    const Stop stop{found[0], found[1] <= found[0] && found[1] < r.drafts};
    __syncthreads();
    return stop;
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

// A cut of the race at the row where a request stops.  Every column's upper
// bound of w / noise, with w = p - q; the column that wins does so for certain
// if its lower bound is above the next upper bound.
template <class E>
__global__ __launch_bounds__(kBlock) void draft_draw_kernel(const DraftArgs a) {
    constexpr int kV = Elem<E>::kVec, kWaves = kBlock / 64;
    __shared__ int found[2];
    __shared__ Race races[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x / a.cuts;
    const int cut = (int)(blockIdx.x - b * a.cuts);
    const Request r = request_of(a, b);
    if (r.drafts < 0) return;
    const Stop stop = stop_of<E, kBlock>(a, r, found);
    if (stop.close) return;                              // finish does it all
    const int64_t at = r.first + stop.end, drafted = r.draft + stop.end;
    const bool refused = stop.end < r.drafts, with_q = refused && a.d;
    const RowSum pr = join_row(a, at, lane);
    RowSum qr{0.0f, 1.0};
    if (with_q) qr = join_row(a, a.R + drafted, lane);
    const int64_t taken = refused && !a.d ? a.ids[drafted] : -1;
    const float pk = (float)((1.0 + kDrawSlack) / pr.s), qk = with_q ? (float)((1.0 - kDrawSlack) / qr.s) : 0.0f;
    const E *x = row_of<E>(a, at), *d = with_q ? row_of<E>(a, a.R + drafted) : x;
    const float *noise = a.noise + b * a.ld_n;
    const float c = a.scale, pm = pr.m, qm = with_q ? qr.m : pr.m;
    const int64_t lo = cut * a.cut, hi = lo + a.cut < a.V ? lo + a.cut : a.V;
    Race v{0.0f, 0.0f, -1};
    for (int64_t col = lo + threadIdx.x * kV; col < hi; col += kBlock * kV) {
        float xs[kV], ds[kV], ns[kV];
        const int64_t n = hi - col;
        load_logits(x + col, n, xs);
        load_logits(d + col, n, ds);
        if (n >= kV) {
#pragma unroll
            for (int i = 0; i < kV; i += 4) Elem<float>::unpack(load16(noise + col + i), ns + i);
        } else {
            load_head<kV>(noise + col, (int)n, 1.0f, ns);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float p = __builtin_amdgcn_exp2f((xs[i] - pm) * c) * pk;
            const float q = __builtin_amdgcn_exp2f((ds[i] - qm) * c) * qk;
            float t = __builtin_fmaxf(p - q, 0.0f) * __builtin_amdgcn_rcpf(ns[i]);
            t = col + i == taken ? 0.0f : t;
            const bool first = t > v.best;
            v.second = __builtin_fmaxf(v.second, first ? v.best : t);
            v.best = first ? t : v.best;
            v.column = first ? col + i : v.column;
        }
    }
    v = merge_lanes(v);
    if (lane == 0) races[wave] = v;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < kWaves; ++i) merge(v, races[i]);
    races_of(a)[blockIdx.x] = v;
}

// ---------------------------------------------------------------- fp64

constexpr int kWide = 1024;         // threads of finish

__device__ __forceinline__ double sum_block(double v, double (&room)[kWide / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = sum_lanes(v);
    if (lane == 0) room[wave] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kWide / 64; ++i) v += room[i];
    __syncthreads();
    return v;
}

// A row's sum in fp64 over the same maximum
template <class E>
__device__ __forceinline__ RowSum exact_row(const DraftArgs &a, int64_t i, const RowSum &fast, double (&room)[kWide / 64]) {
    const E *x = row_of<E>(a, i);
    double s = 0.0;
    for (int64_t col = threadIdx.x; col < a.V; col += kWide) s += exp2(((double)Elem<E>::get(x[col]) - fast.m) * a.scale64);
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
                                              const RowSum &qr, int64_t taken, Exact (&room)[kWide / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const E *x = row_of<E>(a, at), *d = q_at < 0 ? x : row_of<E>(a, q_at);
    Exact v{0.0, -1};
    for (int64_t col = threadIdx.x; col < a.V; col += kWide) {
        double w = share(a, Elem<E>::get(x[col]), pr);
        if (q_at >= 0) w -= share(a, Elem<E>::get(d[col]), qr);
        const double score = w / (double)a.noise[b * a.ld_n + col];
        if (w > 0.0 && score > 0.0 && col != taken) better(v, Exact{score, col});
    }
#pragma unroll
    for (int n = 1; n < 64; n <<= 1) better(v, Exact{__shfl_xor(v.score, n, 64), __shfl_xor(v.column, n, 64)});
    if (lane == 0) room[wave] = v;
    __syncthreads();
    v = room[0];
    for (int i = 1; i < kWide / 64; ++i) better(v, room[i]);
    __syncthreads();
    return v.column;
}

// One block a request
template <class E>
__global__ __launch_bounds__(kWide) void draft_finish_kernel(const DraftArgs a) {
    __shared__ int found[2];
    __shared__ double sums[kWide / 64];
    __shared__ Exact exacts[kWide / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x;
    const Request r = request_of(a, b);
    if (r.drafts < 0) {
        if (threadIdx.x == 0) a.accepted[b] = 0;
        return;
    }
    Stop stop = stop_of<E, kWide>(a, r, found);
    if (stop.close) {                                    // one after another, the close ones in fp64
        for (stop.end = 0; stop.end < r.drafts; ++stop.end) {
            const int64_t row = r.first + stop.end, drafted = r.draft + stop.end;
            RowSum p = join_row(a, row, lane), q{0.0f, 1.0};
            if (a.d) q = join_row(a, a.R + drafted, lane);
            Stand s = stand_of<E>(a, r, stop.end, p, q);
            if (s.close) {
                p = exact_row<E>(a, row, p, sums);
                if (a.d) q = exact_row<E>(a, a.R + drafted, q, sums);
                s = stand_of<E>(a, r, stop.end, p, q);
            }
            if (!s.stands) break;
        }
    }
    const int64_t at = r.first + stop.end, drafted = r.draft + stop.end;
    const bool refused = stop.end < r.drafts, with_q = refused && a.d;
    RowSum pr = join_row(a, at, lane), qr{0.0f, 1.0};
    const RowSum fast = pr;
    if (with_q) qr = join_row(a, a.R + drafted, lane);
    const int64_t taken = refused && !a.d ? a.ids[drafted] : -1;
    int64_t token = -1;
    if (pr.s == pr.s) {                                  // the row has a distribution
        bool certain = false;
        if (!stop.close) {
            Race v{0.0f, 0.0f, -1};
            for (int i = lane; i < a.cuts; i += 64) merge(v, races_of(a)[b * a.cuts + i]);
            v = merge_lanes(v);
            if (v.column >= 0) {
                const double p = share(a, Elem<E>::get(row_of<E>(a, at)[v.column]), pr);
                const double q = with_q ? share(a, Elem<E>::get(row_of<E>(a, a.R + drafted)[v.column]), qr) : 0.0;
                const double lower = ((1.0 - kDrawSlack) * p - (1.0 + kDrawSlack) * q) / (double)a.noise[b * a.ld_n + v.column];
                certain = (double)v.second < lower;
                token = v.column;
            }
        }
        if (!certain) {                                  // uniform: every wave has joined the same races
            pr = exact_row<E>(a, at, pr, sums);
            if (with_q) qr = exact_row<E>(a, a.R + drafted, qr, sums);
            token = exact_race<E>(a, b, at, pr, with_q ? a.R + drafted : -1, qr, taken, exacts);
            if (token < 0 && refused) token = exact_race<E>(a, b, at, pr, -1, qr, -1, exacts);
        }
    }
    if (threadIdx.x == 0) a.accepted[b] = stop.end;
    for (int i = wave; i <= r.drafts; i += kWide / 64) {
        const int64_t row = r.first + i;
        const int64_t id = i < stop.end ? a.ids[r.draft + i] : i == stop.end ? token : -1;
        const RowSum p = i < stop.end ? join_row(a, row, lane) : fast;
        if (lane == 0) {
            float logp = i == stop.end ? __builtin_nanf("") : 0.0f;
            if (id >= 0) logp = (float)(((double)Elem<E>::get(row_of<E>(a, row)[id]) - p.m) * a.inv_temperature - log(p.s));
            a.tokens[row] = id;
            a.logprobs[row] = logp;
        }
    }
}

template <class E, bool ONCE>
void start_rows(const DraftArgs &a, int cus, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.rows * a.slices);
    if (a.rows >= 4 * cus && a.slice <= 8192) draft_rows_kernel<E, 64, ONCE><<<grid, 64, 0, stream>>>(a);
    else if (a.slice <= 65536) draft_rows_kernel<E, kBlock, ONCE><<<grid, kBlock, 0, stream>>>(a);
    else draft_rows_kernel<E, 1024, ONCE><<<grid, 1024, 0, stream>>>(a);
}
template <class E>
void start(const DraftArgs &a, int cus, hipStream_t stream) {
    start_rows<E, false>(a, cus, stream);
    draft_draw_kernel<E><<<(unsigned)(a.B * a.cuts), kBlock, 0, stream>>>(a);
    draft_finish_kernel<E><<<(unsigned)a.B, kWide, 0, stream>>>(a);
}

}  // namespace

DraftCut draft_cut(int64_t rows, int64_t B, int64_t V, int cus) {
    // slices of a row: one where the rows alone give every compute unit a block, else enough for four blocks each
    int64_t slices = 1;
    if (rows < cus) {
        const int64_t want = ceil_div((int64_t)cus * 4, rows), most = ceil_div(V, 4096);
        slices = want < most ? want : most;
    }
    // cuts of a race: four blocks for every compute unit, of at least 2048 columns
    const int64_t want = ceil_div((int64_t)cus * 4, B), most = ceil_div(V, 2048);
    const int64_t cuts = want < most ? want : most;
    return {(int)slices, (int)cuts, ceil_div(ceil_div(V, slices), 8) * 8, ceil_div(ceil_div(V, cuts), 8) * 8,
            rows * slices * (int64_t)sizeof(Part) + B * cuts * (int64_t)sizeof(Race)};
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
