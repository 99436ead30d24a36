// C ABI of the gated activation with an 8-bit checkpoint, the low-rank
// adapters and the verification of drafted tokens: argument validation and
// dispatch.  The contract of every entry point is documented in
// include/mxfp8_policy.h.
#include "mxfp8_policy.h"

#include <hip/hip_runtime.h>

#include "mx_api.hpp"
#include "mx_launch.hpp"
#include "mx_spans.hpp"

using namespace mx;

namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;
constexpr int64_t kMaxElements = (int64_t)1 << 60;

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// rows of `cols` elements ld apart, with byte offsets that fit 63 bits
bool rows_ok(int64_t T, int64_t cols, int64_t ld) { return ld >= cols && (T == 0 || ld <= kMaxElements / T); }

bool swiglu_sizes_ok(int64_t T, int64_t I) {
    return T >= 0 && T < kMaxInt && I >= 32 && I % 32 == 0 && I < ((int64_t)1 << 30) &&
           (T == 0 || I <= (((int64_t)1 << 35) - 1) / T);
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

bool lora_sizes_ok(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N) {
    return rows >= 0 && rows < kMaxInt && rows % 32 == 0 && E >= 1 && E <= kLoraMaxAdapters && r >= 8 &&
           r <= kLoraMaxRank && r % 8 == 0 && K >= 8 && K < kMaxInt && K % 8 == 0 && N >= 8 && N < kMaxInt && N % 8 == 0 &&
           rows / 32 * ceil_div(K > N ? K : N, 256) < ((int64_t)1 << 24) &&
           (rows / 256 + E) * ceil_div(K + N, 128) < ((int64_t)1 << 22) && E * r * (K + N) < ((int64_t)1 << 40);
}

bool drafts_sizes_ok(int64_t R, int64_t B, int64_t V) {
    return B >= 0 && R >= B && R < kMaxInt && V >= 1 && V < kMaxInt && (2 * R - B) * ceil_div(V, 4096) < ((int64_t)1 << 22);
}

// The parts of a workspace, in order, each from a multiple of 256 bytes on.
struct Parts {
    int64_t at = 0;
    int64_t take(int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    }
};
struct LoraBackwardParts {
    LoraCut cut;
    LoraOuterPlan plan;
    int64_t at, bt, part, s, h, slots_a, slots_b, total;
};
LoraBackwardParts lora_backward_parts(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N) {
    LoraBackwardParts w{};
    const int cus = device_cu_count();
    w.cut = lora_cut(rows, N, cus);
    w.plan = lora_outer_plan(rows, E, r, K, N, cus);
    Parts p;
    w.at = p.take(E * r * K * 2), w.bt = p.take(E * r * N * 2);
    w.part = p.take(w.cut.splits * rows * r * 4);
    w.s = p.take(lora_packed_bytes(rows, r)), w.h = p.take(lora_packed_bytes(rows, r));
    w.slots_a = p.take(w.plan.slots * r * K * 4), w.slots_b = p.take(w.plan.slots * r * N * 4);
    w.total = p.at;
    return w;
}

}  // namespace

extern "C" {

mxfp8_status mxfp8_swiglu(const void *gu, int64_t ld, int64_t T, int64_t I, void *h, uint8_t *h_q, uint8_t *h_s,
                          mxfp8_layout h_layout, uint8_t *saved_q, uint8_t *saved_s, hipStream_t stream) {
    const bool packed = raw(h_layout) == MXFP8_PACKED;
    if (!packed && raw(h_layout) != MXFP8_CANONICAL) return MXFP8_ERR_DTYPE;
    if (!swiglu_sizes_ok(T, I) || !rows_ok(T, 2 * I, ld) || ld % 8) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!gu || (h && (h_q || h_s)) || (!h && (!h_q || !h_s)) || !saved_q != !saved_s) return MXFP8_ERR_NULL;
    if (h_q && packed && mxfp8_packed_bytes(1, T, I, 0) == 0) return MXFP8_ERR_SHAPE;
    for (const void *p : {gu, (const void *)h, (const void *)h_q, (const void *)h_s, (const void *)saved_q, (const void *)saved_s})
        if (!aligned(p, 16)) return MXFP8_ERR_ALIGN;
    const int64_t n = T * I;
    const int64_t hq_bytes = packed ? packed_q_bytes(1, T, I) : n, hs_bytes = packed ? packed_s_bytes(1, T, I) : n / 32;
    if (overlap({{h, n * 2}, {h_q, hq_bytes}, {h_s, hs_bytes}, {saved_q, n * 2}, {saved_s, n / 16}},
                {{gu, T, 4 * I, 2 * ld}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    SwigluArgs a{};
    a.x = static_cast<const uint16_t *>(gu), a.ld = ld, a.T = T, a.I = (int)I, a.h = static_cast<uint16_t *>(h);
    a.hq = h_q, a.hs = h_s, a.q = saved_q, a.s = saved_s;
    return finish(launch_swiglu(a, packed, stream));
}

mxfp8_status mxfp8_swiglu_backward(const void *d_h, int64_t ld, int64_t T, int64_t I, const uint8_t *saved_q,
                                   const uint8_t *saved_s, void *d_gu, void *h, hipStream_t stream) {
    if (!swiglu_sizes_ok(T, I) || !rows_ok(T, I, ld) || ld % 8) return MXFP8_ERR_SHAPE;
    if (T == 0) return MXFP8_OK;
    if (!d_h || !saved_q || !saved_s || !d_gu) return MXFP8_ERR_NULL;
    if (h == d_h && ld != I && T > 1) return MXFP8_ERR_SHAPE;
    for (const void *p : {d_h, (const void *)saved_q, (const void *)saved_s, (const void *)d_gu, (const void *)h})
        if (!aligned(p, 16)) return MXFP8_ERR_ALIGN;
    const int64_t n = T * I;
    // a lane reads the values of d_h at the places of h that it alone writes
    if (overlap({{d_gu, n * 4}, {h, n * 2}},
                {{h == d_h ? nullptr : d_h, T, 2 * I, 2 * ld}, {saved_q, n * 2}, {saved_s, n / 16}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    SwigluArgs a{};
    a.x = static_cast<const uint16_t *>(d_h), a.ld = ld, a.T = T, a.I = (int)I, a.h = static_cast<uint16_t *>(h);
    a.q = const_cast<uint8_t *>(saved_q), a.s = const_cast<uint8_t *>(saved_s), a.dx = static_cast<uint16_t *>(d_gu);
    return finish(launch_swiglu_backward(a, stream));
}

size_t mxfp8_lora_add_workspace_bytes(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N) {
    if (!lora_sizes_ok(rows, E, r, K, N)) return 0;
    return (size_t)round_up(lora_cut(rows, K, device_cu_count()).splits * rows * r * 4, 256);
}

mxfp8_status mxfp8_lora_add(void *y, mxfp8_dtype y_dtype, int64_t ld_y, const void *x, int64_t ld_x, int64_t T,
                            const void *a, const void *b, const float *scales, int64_t E, int64_t r, int64_t K,
                            int64_t N, const int32_t *offsets, const int64_t *row_token, int64_t rows, float *hidden,
                            void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (raw(y_dtype) != MXFP8_F32 && raw(y_dtype) != MXFP8_BF16) return MXFP8_ERR_DTYPE;
    const int64_t e = raw(y_dtype) == MXFP8_BF16 ? 2 : 4;
    if (!lora_sizes_ok(rows, E, r, K, N) || T < 0 || T >= kMaxInt || !rows_ok(T, N, ld_y) || !rows_ok(T, K, ld_x) || ld_y % 8 || ld_x % 8)
        return MXFP8_ERR_SHAPE;
    if (rows == 0) return MXFP8_OK;
    const int64_t need = (int64_t)mxfp8_lora_add_workspace_bytes(rows, E, r, K, N);
    if ((T && (!y || !x)) || !a || !b || !offsets || !row_token || !workspace) return MXFP8_ERR_NULL;
    if ((int64_t)workspace_bytes < need) return MXFP8_ERR_SHAPE;
    for (const void *p : {(const void *)y, x, a, b, (const void *)hidden, (const void *)workspace})
        if (!aligned(p, 16)) return MXFP8_ERR_ALIGN;
    if (!aligned(scales, 4) || !aligned(offsets, 4) || !aligned(row_token, 8)) return MXFP8_ERR_ALIGN;
    if (overlap({{y, T, N * e, ld_y * e}, {hidden, rows * r * 4}, {workspace, need}},
                {{x, T, K * 2, ld_x * 2}, {a, E * r * K * 2}, {b, E * N * r * 2}, {scales, E * 4}, {offsets, (E + 1) * 4}, {row_token, rows * 8}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    const LoraCut cut = lora_cut(rows, K, device_cu_count());
    LoraShrink s{};
    s.x = static_cast<const uint16_t *>(x), s.ld = ld_x, s.T = T, s.w = static_cast<const uint16_t *>(a);
    s.offsets = offsets, s.row_token = row_token, s.rows = rows, s.part = static_cast<float *>(workspace);
    s.E = (int)E, s.r = (int)r, s.K = (int)K, s.splits = cut.splits, s.slice = cut.slice;
    LoraExpand p{};
    p.y = y, p.ld = ld_y, p.T = T, p.w = static_cast<const uint16_t *>(b), p.scales = scales, p.offsets = offsets;
    p.row_token = row_token, p.rows = rows, p.part = s.part, p.hidden = hidden;
    p.E = T ? (int)E : 0, p.r = (int)r, p.N = T ? (int)N : 0, p.splits = cut.splits;
    if (T && lora_both(rows, T, r, K, device_cu_count())) return finish(launch_lora_both(s, p, e == 2, stream));
    if (T) st = finish(launch_lora_shrink(s, stream));
    if (st != MXFP8_OK) return st;
    return finish(launch_lora_expand(p, e == 2, stream));
}

size_t mxfp8_lora_backward_workspace_bytes(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N) {
    if (!lora_sizes_ok(rows, E, r, K, N)) return 0;
    return (size_t)lora_backward_parts(rows, E, r, K, N).total;
}

mxfp8_status mxfp8_lora_backward(void *d_x, int64_t ld_dx, const void *d_y, int64_t ld_dy, const void *x,
                                 const uint8_t *x_s, mxfp8_input x_input, int64_t ld_x, int64_t T, const void *a,
                                 const void *b, const float *scales, int64_t E, int64_t r, int64_t K, int64_t N,
                                 const int32_t *offsets, const int64_t *row_token, int64_t rows, const float *hidden,
                                 float *d_a, float *d_b, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
    const int form = raw(x_input);
    if (form != MXFP8_INPUT_BF16 && form != MXFP8_INPUT_CANONICAL && form != MXFP8_INPUT_PACKED) return MXFP8_ERR_DTYPE;
    const bool grid = form != MXFP8_INPUT_BF16, packed = form == MXFP8_INPUT_PACKED;
    if (!lora_sizes_ok(rows, E, r, K, N) || T < 0 || T >= kMaxInt || !rows_ok(T, N, ld_dy) || ld_dy % 8) return MXFP8_ERR_SHAPE;
    if (d_x && (!rows_ok(T, K, ld_dx) || ld_dx % 8)) return MXFP8_ERR_SHAPE;
    if (grid ? K % 32 != 0 || (packed && T && mxfp8_packed_bytes(1, T, K, 0) == 0) : !rows_ok(T, K, ld_x) || ld_x % 8) return MXFP8_ERR_SHAPE;
    const int64_t used = T ? rows : 0;                   // without tokens every row is padding
    const LoraBackwardParts w = lora_backward_parts(rows, E, r, K, N);
    if ((used && (!d_y || !x || (grid && !x_s) || !row_token || !hidden)) || !a || !b || !offsets || !d_a || !d_b || !workspace)
        return MXFP8_ERR_NULL;
    if ((int64_t)workspace_bytes < w.total) return MXFP8_ERR_SHAPE;
    for (const void *p : {(const void *)d_x, d_y, x, (const void *)x_s, a, b, (const void *)hidden, (const void *)d_a, (const void *)d_b,
                          (const void *)workspace})
        if (!aligned(p, 16)) return MXFP8_ERR_ALIGN;
    if (!aligned(scales, 4) || !aligned(offsets, 4) || !aligned(row_token, 8)) return MXFP8_ERR_ALIGN;
    const Span xs = !grid ? Span(x, T, K * 2, ld_x * 2) : packed ? Span(x, packed_q_bytes(1, T, K)) : Span(x, T * K);
    const Span ss = !grid ? Span(nullptr, 0) : packed ? Span(x_s, packed_s_bytes(1, T, K)) : Span(x_s, T * K / 32);
    if (overlap({{d_x, T, K * 2, ld_dx * 2}, {d_a, E * r * K * 4}, {d_b, E * N * r * 4}, {workspace, w.total}},
                {{d_y, T, N * 2, ld_dy * 2}, xs, ss, {a, E * r * K * 2}, {b, E * N * r * 2}, {scales, E * 4}, {offsets, (E + 1) * 4},
                 {row_token, rows * 8}, {hidden, rows * r * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    char *base = static_cast<char *>(workspace);
    LoraVec *s_rows = reinterpret_cast<LoraVec *>(base + w.s), *h_rows = reinterpret_cast<LoraVec *>(base + w.h);
    if (used) {
        LoraPrepare t{};
        t.hidden = hidden, t.packed = h_rows, t.scales = scales, t.offsets = offsets, t.row_token = row_token;
        t.rows = rows, t.T = T, t.E = (int)E, t.r = (int)r;
        t.job[0] = {static_cast<const uint16_t *>(a), reinterpret_cast<uint16_t *>(base + w.at), (int)r, (int)K};
        t.job[1] = {static_cast<const uint16_t *>(b), reinterpret_cast<uint16_t *>(base + w.bt), (int)N, (int)r};
        st = finish(launch_lora_prepare(t, stream));
        if (st != MXFP8_OK) return st;
        LoraShrink s{};
        s.x = static_cast<const uint16_t *>(d_y), s.ld = ld_dy, s.T = T, s.w = t.job[1].to, s.offsets = offsets;
        s.row_token = row_token, s.rows = rows, s.part = reinterpret_cast<float *>(base + w.part);
        s.E = (int)E, s.r = (int)r, s.K = (int)N, s.splits = w.cut.splits, s.slice = w.cut.slice;
        LoraExpand p{};
        p.y = d_x, p.ld = ld_dx, p.T = T, p.w = t.job[0].to, p.scales = scales, p.offsets = offsets;
        p.row_token = row_token, p.rows = rows, p.part = s.part, p.packed = s_rows;
        p.E = (int)E, p.r = (int)r, p.N = d_x ? (int)K : 0, p.splits = w.cut.splits;
        if (lora_both(rows, T, r, N, device_cu_count())) {
            st = finish(launch_lora_both(s, p, true, stream));
        } else {
            st = finish(launch_lora_shrink(s, stream));
            if (st != MXFP8_OK) return st;
            st = finish(launch_lora_expand(p, true, stream));
        }
        if (st != MXFP8_OK) return st;
    }
    LoraOuter o{};
    o.wide[0] = {s_rows, x, x_s, grid ? K : ld_x, packed_ksteps(K), (int)K, d_a, reinterpret_cast<float *>(base + w.slots_a), 0};
    o.wide[1] = {h_rows, d_y, nullptr, ld_dy, 0, (int)N, d_b, reinterpret_cast<float *>(base + w.slots_b), 0};
    o.offsets = offsets, o.row_token = row_token, o.rows = used, o.T = T, o.E = (int)E, o.r = (int)r;
    return finish(launch_lora_outer(o, w.plan, form, stream));
}

size_t mxfp8_verify_drafts_workspace_bytes(int64_t R, int64_t B, int64_t V, int draft_logits) {
    if (!drafts_sizes_ok(R, B, V) || B == 0) return 0;
    return (size_t)draft_cut(draft_logits ? 2 * R - B : R, B, V, device_cu_count()).bytes;
}

mxfp8_status mxfp8_verify_drafts(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t R, int64_t V,
                                 const int32_t *offsets, int64_t B, const int64_t *draft_ids, const float *uniforms,
                                 const void *draft_logits, int64_t ld_draft, const float *noise, int64_t ld_noise,
                                 double temperature, int32_t *accepted, int64_t *tokens, float *logprobs,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (raw(dtype) != MXFP8_F32 && raw(dtype) != MXFP8_BF16) return MXFP8_ERR_DTYPE;
    if (!drafts_sizes_ok(R, B, V) || !rows_ok(R, V, ld) || !rows_ok(B, V, ld_noise)) return MXFP8_ERR_SHAPE;
    const int64_t D = R - B, e = raw(dtype) == MXFP8_BF16 ? 2 : 4;
    if (draft_logits && !rows_ok(D, V, ld_draft)) return MXFP8_ERR_SHAPE;
    if (!(temperature >= 0x1p-60 && temperature <= 0x1p60)) return MXFP8_ERR_SHAPE;
    if (B == 0) return MXFP8_OK;
    if (!logits || !offsets || !noise || !accepted || !tokens || !logprobs || !workspace || (D && (!draft_ids || !uniforms)))
        return MXFP8_ERR_NULL;
    const void *draft = D ? draft_logits : nullptr;
    const int64_t rows = draft ? R + D : R, need = draft_cut(rows, B, V, device_cu_count()).bytes;
    if ((int64_t)workspace_bytes < need) return MXFP8_ERR_SHAPE;
    if (!aligned(logits, e) || !aligned(draft_logits, e) || !aligned(offsets, 4) || !aligned(draft_ids, 8) || !aligned(uniforms, 4) ||
        !aligned(noise, 4) || !aligned(accepted, 4) || !aligned(tokens, 8) || !aligned(logprobs, 4) || !aligned(workspace, 16))
        return MXFP8_ERR_ALIGN;
    if (overlap({{accepted, B * 4}, {tokens, R * 8}, {logprobs, R * 4}, {workspace, need}},
                {{logits, R, V * e, ld * e}, {draft, D, V * e, ld_draft * e}, {offsets, (B + 1) * 4}, {draft_ids, D * 8},
                 {uniforms, D * 4}, {noise, B, V * 4, ld_noise * 4}}))
        return MXFP8_ERR_OVERLAP;
    mxfp8_status st = check_device();
    if (st != MXFP8_OK) return st;
    DraftArgs a{};
    a.x = logits, a.ld = ld, a.R = R, a.V = V, a.B = B, a.offsets = offsets, a.ids = draft_ids, a.u = uniforms;
    a.d = draft, a.ld_d = ld_draft, a.noise = noise, a.ld_n = ld_noise, a.temperature = temperature;
    a.accepted = accepted, a.tokens = tokens, a.logprobs = logprobs, a.workspace = workspace, a.rows = rows;
    return finish(launch_drafts(a, e == 2, stream));
}

}  // extern "C"
