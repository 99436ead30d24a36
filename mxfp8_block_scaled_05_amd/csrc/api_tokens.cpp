// C ABI of the token-level operators: argument validation and dispatch.  The
// contract of every entry point is documented in include/mxfp8_tokens.h.
#include "mxfp8_tokens.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "mx_api.hpp"
#include "mx_launch.hpp"

using namespace mx;

namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;

// a * b < 2^31 for a, b >= 0
bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= (kMaxInt - 1) / a; }
// rows of `cols` elements ld apart, with byte offsets that fit 63 bits
bool rows_ok(int64_t T, int64_t cols, int64_t ld) { return ld >= cols && (T == 0 || ld <= ((int64_t)1 << 60) / T); }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(const mxfp8_dtype &d) { return raw(d) == MXFP8_F32 || raw(d) == MXFP8_BF16; }
bool score_ok(const mxfp8_score &s) { return raw(s) == MXFP8_SCORE_SOFTMAX || raw(s) == MXFP8_SCORE_SIGMOID; }
size_t elem_bytes(const mxfp8_dtype &d) { return raw(d) == MXFP8_BF16 ? 2 : 4; }

bool temperature_ok(double t) { return t >= 0x1p-60 && t <= 0x1p60; }   // 1 / t stays an fp32 number
// workgroups of 256 threads whose threads must stay below 2^32
bool grid_ok(int64_t blocks) { return blocks < ((int64_t)1 << 24); }

bool route_sizes_ok(int64_t ld, int64_t T, int64_t E, int64_t k) {
    return T >= 0 && T < kMaxInt && E >= 1 && E <= kRouteMaxExperts && k >= 1 && k <= kRouteMaxK && k <= E &&
           rows_ok(T, E, ld) && grid_ok(ceil_div(T, 4));
}

// A buffer: `rows` rows of `bytes` bytes, `step` bytes apart.
struct Span {
    uintptr_t at;
    int64_t rows, bytes, step;
    Span(const void *p, int64_t n) : at((uintptr_t)p), rows(1), bytes(n), step(n) {}
    Span(const void *p, int64_t rows_, int64_t n, int64_t step_) : at((uintptr_t)p), rows(rows_), bytes(n), step(step_) {}
    bool empty() const { return !at || rows <= 0 || bytes <= 0; }
    uintptr_t end() const { return at + (rows - 1) * step + bytes; }
};

// Whether rows of a and b, both step bytes apart, share a byte: b's row j meets
// a's row i if j - i lies between two bounds that follow from the distance.
bool rows_meet(const Span &a, const Span &b, int64_t step) {
    const int64_t d = (int64_t)(a.at - b.at);
    const int64_t above = d - b.bytes, below = d + a.bytes;          // above < (j - i) * step < below
    const int64_t lo = above >= 0 ? above / step + 1 : -((-above - 1) / step);
    const int64_t hi = below > 0 ? (below - 1) / step : -(-below / step) - 1;
    return (lo > 1 - a.rows ? lo : 1 - a.rows) <= (hi < b.rows - 1 ? hi : b.rows - 1);
}
bool meet(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
    if (a.rows == 1 || a.step == b.step) return rows_meet(a, b, b.step);
    if (b.rows == 1) return rows_meet(b, a, a.step);
    if (a.rows > b.rows) return meet(b, a);
    for (int64_t i = 0; i < a.rows; ++i)
        if (rows_meet(Span(reinterpret_cast<const void *>(a.at + i * a.step), a.bytes), b, b.step)) return true;
    return false;
}

// Whether an output shares a byte with an input or with another output.
bool overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (meet(*o, i)) return true;
        for (const Span *q = o + 1; q != outputs.end(); ++q)
            if (meet(*o, *q)) return true;
    }
    return false;
}

}  // namespace

extern "C" {

mxfp8_status mxfp8_route(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                         mxfp8_score score, const float *bias, int64_t groups, int64_t groups_kept,
                         int64_t group_top, int renormalize, float scale, int32_t *ids, float *weights,
                         hipStream_t stream) {
    if (!dtype_ok(dtype) || !score_ok(score)) return MXFP8_ERR_DTYPE;
    if (!route_sizes_ok(ld, T, E, k)) return MXFP8_ERR_SHAPE;
    if (groups < 1 || groups > kRouteMaxGroups || E % groups || groups_kept < 1 || groups_kept > groups)
        return MXFP8_ERR_SHAPE;
    const int64_t size = E / groups;
    if (group_top < 1 || group_top > 2 || group_top > size || k > groups_kept * size) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!logits || !ids || !weights) return MXFP8_ERR_NULL;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return MXFP8_ERR_ALIGN;
    const int64_t e = elem_bytes(dtype);
    if (overlap({{ids, T * k * 4}, {weights, T * k * 4}}, {{logits, T, E * e, ld * e}, {bias, E * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    RouteArgs a{};
    a.x = logits, a.ld = ld, a.T = T, a.bias = bias, a.ids = ids, a.w = weights, a.scale = scale;
    a.E = (int)E, a.k = (int)k, a.groups = (int)groups, a.size = (int)size, a.kept = (int)groups_kept;
    a.group_top = (int)group_top, a.sigmoid = raw(score) == MXFP8_SCORE_SIGMOID, a.renorm = renormalize != 0;
    return finish(launch_route(a, raw(dtype) == MXFP8_BF16, stream));
}

mxfp8_status mxfp8_route_backward(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t E,
                                  int64_t k, mxfp8_score score, const int32_t *ids, const float *d_weights,
                                  int renormalize, float scale, void *d_logits, hipStream_t stream) {
    if (!dtype_ok(dtype) || !score_ok(score)) return MXFP8_ERR_DTYPE;
    if (!route_sizes_ok(ld, T, E, k)) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!logits || !ids || !d_weights || !d_logits) return MXFP8_ERR_NULL;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(d_logits, elem_bytes(dtype)) || !aligned(ids, 4) ||
        !aligned(d_weights, 4))
        return MXFP8_ERR_ALIGN;
    const int64_t e = elem_bytes(dtype);
    if (overlap({{d_logits, T * E * e}}, {{logits, T, E * e, ld * e}, {ids, T * k * 4}, {d_weights, T * k * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    RouteArgs a{};
    a.x = logits, a.ld = ld, a.T = T, a.ids = const_cast<int32_t *>(ids), a.dw = d_weights, a.dx = d_logits;
    a.scale = scale, a.E = (int)E, a.k = (int)k, a.sigmoid = raw(score) == MXFP8_SCORE_SIGMOID;
    a.renorm = renormalize != 0;
    return finish(launch_route_backward(a, raw(dtype) == MXFP8_BF16, stream));
}

int64_t mxfp8_route_rows(int64_t pairs, int64_t E, int64_t pad) {
    if (pairs < 0 || pairs >= kMaxInt || E < 1 || E > kTablesMaxExperts || pad < 1 || pad > 1024) return 0;
    const int64_t used = E < pairs ? E : pairs;
    return (pairs + used * (pad - 1)) / pad * pad;
}

size_t mxfp8_route_tables_workspace_bytes(int64_t T, int64_t k, int64_t E) {
    if (T < 1 || k < 1 || T >= kMaxInt || !product_ok(T, k) || E < 1 || E > kTablesMaxExperts) return 0;
    return (size_t)route_tables_workspace_bytes(T * k, E);
}

mxfp8_status mxfp8_route_tables(const int32_t *ids, int64_t T, int64_t k, int64_t E, int64_t pad,
                                int32_t *offsets, int32_t *counts, int64_t *row_token, int64_t rows,
                                int32_t *pair_row, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!ids || !offsets || !counts || !row_token || !pair_row) return MXFP8_ERR_NULL;
    if (T < 1 || k < 1 || T >= kMaxInt || !product_ok(T, k) || E < 1 || E > kTablesMaxExperts || pad < 1 || pad > 1024)
        return MXFP8_ERR_SHAPE;
    if (T * k + E * pad >= kMaxInt || rows >= kMaxInt || rows < mxfp8_route_rows(T * k, E, pad)) return MXFP8_ERR_SHAPE;
    const size_t need = mxfp8_route_tables_workspace_bytes(T, k, E);
    if (need && !workspace) return MXFP8_ERR_NULL;
    if (workspace_bytes < need) return MXFP8_ERR_SHAPE;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(row_token, 8) ||
        !aligned(pair_row, 4) || !aligned(workspace, 4))
        return MXFP8_ERR_ALIGN;
    const int64_t pairs = T * k;
    if (overlap({{offsets, (E + 1) * 4}, {counts, E * 4}, {row_token, rows * 8}, {pair_row, pairs * 4}, {workspace, (int64_t)need}},
                {{ids, pairs * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    RouteTables a{};
    a.ids = ids, a.offsets = offsets, a.counts = counts, a.pair_row = pair_row, a.row_token = row_token;
    a.hist = static_cast<int32_t *>(workspace), a.pairs = T * k, a.rows = rows;
    a.k = (int)k, a.E = (int)E, a.pad = (int)pad;
    return finish(launch_route_tables(a, stream));
}

static mxfp8_status combine_sizes(int64_t rows, int64_t H, int64_t T, int64_t k) {
    if (rows < 0 || rows >= kMaxInt || H < 1 || H >= kMaxInt || T < 0 || T >= kMaxInt || k < 1 || !product_ok(T, k) ||
        !rows_ok(rows, H, H))
        return MXFP8_ERR_SHAPE;
    // a thread per 4 elements of an output row; a wave per pair and per 8 rows
    if (!product_ok(T, ceil_div(H, 4)) || !grid_ok(ceil_div(T * ceil_div(H, 4), 256)) ||
        !grid_ok(ceil_div(T * k, 4) + ceil_div(rows, 32)))
        return MXFP8_ERR_SHAPE;
    return MXFP8_OK;
}

mxfp8_status mxfp8_moe_combine(const void *y, mxfp8_dtype dtype, int64_t rows, int64_t H, const int32_t *pair_row,
                               const float *weights, int64_t T, int64_t k, void *out, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MXFP8_ERR_DTYPE;
    mxfp8_status st = combine_sizes(rows, H, T, k);
    if (st != MXFP8_OK) return st;
    if (T == 0) return MXFP8_OK;
    if ((!y && rows) || !pair_row || !weights || !out) return MXFP8_ERR_NULL;
    if (!aligned(y, elem_bytes(dtype)) || !aligned(out, elem_bytes(dtype)) || !aligned(pair_row, 4) ||
        !aligned(weights, 4))
        return MXFP8_ERR_ALIGN;
    const int64_t line = H * (int64_t)elem_bytes(dtype);
    if (overlap({{out, T, line, line}}, {{y, rows, line, line}, {pair_row, T * k * 4}, {weights, T * k * 4}}))
        return MXFP8_ERR_OVERLAP;
    st = check_device();
    if (st != MXFP8_OK) return st;
    CombineArgs a{};
    a.y = y, a.pair_row = pair_row, a.w = weights, a.out = out, a.T = T, a.rows = rows, a.H = H, a.k = (int)k;
    return finish(launch_combine(a, raw(dtype) == MXFP8_BF16, stream));
}

mxfp8_status mxfp8_moe_combine_backward(const void *d_out, const void *y, mxfp8_dtype dtype, int64_t rows, int64_t H,
                                        const int32_t *pair_row, const float *weights, const int64_t *row_token,
                                        int64_t T, int64_t k, void *d_y, float *d_weights, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MXFP8_ERR_DTYPE;
    mxfp8_status st = combine_sizes(rows, H, T, k);
    if (st != MXFP8_OK) return st;
    if (T == 0 && rows == 0) return MXFP8_OK;
    if (T > 0 && (!d_out || !pair_row || !weights || !d_weights)) return MXFP8_ERR_NULL;
    if (rows > 0 && (!y || !row_token || !d_y)) return MXFP8_ERR_NULL;
    const size_t e = elem_bytes(dtype);
    if (!aligned(d_out, e) || !aligned(y, e) || !aligned(d_y, e) || !aligned(pair_row, 4) || !aligned(weights, 4) ||
        !aligned(d_weights, 4) || !aligned(row_token, 8))
        return MXFP8_ERR_ALIGN;
    // a pair's row of y and its weight are read by the lanes that write its row of d_y and its d_weights alone
    const int64_t line = H * (int64_t)e, pairs = T * k;
    if (overlap({{d_y, rows, line, line}, {d_weights, pairs * 4}},
                {{y == d_y ? nullptr : y, rows, line, line}, {weights == d_weights ? nullptr : weights, pairs * 4},
                 {d_out, T, line, line}, {pair_row, pairs * 4}, {row_token, rows * 8}}))
        return MXFP8_ERR_OVERLAP;
    st = check_device();
    if (st != MXFP8_OK) return st;
    CombineArgs a{};
    a.y = y, a.pair_row = pair_row, a.w = weights, a.d_out = d_out, a.row_token = row_token, a.d_y = d_y;
    a.d_w = d_weights, a.T = T, a.rows = rows, a.H = H, a.k = (int)k;
    return finish(launch_combine_backward(a, raw(dtype) == MXFP8_BF16, stream));
}

static bool logprobs_sizes_ok(int64_t T, int64_t V) {
    return T >= 0 && T < kMaxInt && V >= 1 && V < kMaxInt && product_ok(T, ceil_div(V, 4096)) &&
           grid_ok(T * ceil_div(V, 4096));
}

size_t mxfp8_token_logprobs_workspace_bytes(int64_t T, int64_t V, int64_t top_n) {
    if (!logprobs_sizes_ok(T, V) || T == 0 || top_n < 0 || top_n > kLogprobsMaxTop || top_n > V) return 0;
    return (size_t)logprobs_workspace_bytes(T, V, (int)top_n, device_cu_count());
}

mxfp8_status mxfp8_token_logprobs(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t V,
                                  const int64_t *targets, double temperature, int64_t top_n, float *logprobs,
                                  float *entropy, float *stats, float *top_logprobs, int64_t *top_ids,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MXFP8_ERR_DTYPE;
    if (!logprobs_sizes_ok(T, V) || !rows_ok(T, V, ld) || top_n < 0 || top_n > kLogprobsMaxTop || top_n > V)
        return MXFP8_ERR_SHAPE;
    if (!temperature_ok(temperature)) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!logits || !targets || !logprobs || !entropy || !stats || (top_n && (!top_logprobs || !top_ids)))
        return MXFP8_ERR_NULL;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(targets, 8) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
        !aligned(stats, 4) || !aligned(top_logprobs, 4) || !aligned(top_ids, 8) || !aligned(workspace, 16))
        return MXFP8_ERR_ALIGN;
    const int64_t e = elem_bytes(dtype);
    const int64_t used = workspace ? logprobs_workspace_bytes(T, V, (int)top_n, device_cu_count()) : 0;
    if (overlap({{logprobs, T * 4}, {entropy, T * 4}, {stats, T * 8}, {top_logprobs, T * top_n * 4}, {top_ids, T * top_n * 8},
                 {workspace, (int64_t)workspace_bytes < used ? 0 : used}},
                {{logits, T, V * e, ld * e}, {targets, T * 8}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    LogprobsArgs a{};
    a.x = logits, a.ld = ld, a.T = T, a.V = V, a.targets = targets, a.temperature = temperature, a.top = (int)top_n;
    a.logprobs = logprobs, a.entropy = entropy, a.stats = stats, a.top_logprobs = top_logprobs, a.top_ids = top_ids;
    a.workspace = workspace;
    return finish(launch_logprobs(a, raw(dtype) == MXFP8_BF16, workspace_bytes, stream));
}

mxfp8_status mxfp8_token_logprobs_backward(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t V,
                                           const int64_t *targets, const float *stats, const float *entropy,
                                           const float *d_logprobs, const float *d_entropy, double temperature,
                                           void *d_logits, int64_t ld_out, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MXFP8_ERR_DTYPE;
    if (!logprobs_sizes_ok(T, V) || !rows_ok(T, V, ld) || !rows_ok(T, V, ld_out)) return MXFP8_ERR_SHAPE;
    if (!temperature_ok(temperature)) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!logits || !targets || !stats || !d_logits || (!d_logprobs && !d_entropy) || (d_entropy && !entropy))
        return MXFP8_ERR_NULL;
    if (logits == d_logits && ld != ld_out && T > 1) return MXFP8_ERR_SHAPE;
    const size_t e = elem_bytes(dtype);
    if (!aligned(logits, e) || !aligned(d_logits, e) || !aligned(targets, 8) || !aligned(stats, 4) ||
        !aligned(entropy, 4) || !aligned(d_logprobs, 4) || !aligned(d_entropy, 4))
        return MXFP8_ERR_ALIGN;
    if (overlap({{d_logits, T, (int64_t)(V * e), (int64_t)(ld_out * e)}},
                {{logits == d_logits ? nullptr : logits, T, (int64_t)(V * e), (int64_t)(ld * e)}, {targets, T * 8},
                 {stats, T * 8}, {entropy, T * 4}, {d_logprobs, T * 4}, {d_entropy, T * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    LogprobsArgs a{};
    a.x = logits, a.ld = ld, a.T = T, a.V = V, a.targets = targets, a.temperature = temperature;
    a.entropy = const_cast<float *>(entropy), a.stats = const_cast<float *>(stats);
    a.d_logprobs = d_logprobs, a.d_entropy = d_entropy, a.dx = d_logits, a.ld_out = ld_out;
    return finish(launch_logprobs_backward(a, raw(dtype) == MXFP8_BF16, stream));
}

}  // extern "C"
