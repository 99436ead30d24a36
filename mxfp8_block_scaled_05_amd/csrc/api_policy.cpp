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

}  // extern "C"
