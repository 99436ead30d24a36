// BF16 values of a block to E4M3 codes (quantize.hip, swiglu.hip).
#pragma once

#include "mx_device.hpp"

namespace mx {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ us2 as_us2(uint32_t v) { return __builtin_bit_cast(us2, v); }
__device__ __forceinline__ uint32_t as_u32(us2 v) { return __builtin_bit_cast(uint32_t, v); }

// max of the two BF16 magnitudes packed in each dword, over n dwords
__device__ __forceinline__ uint32_t max_mag(const uint32_t *d, int n) {
    us2 m = as_us2(d[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < n; ++i) m = __builtin_elementwise_max(m, as_us2(d[i] & 0x7FFF7FFFu));
    return m.x > m.y ? m.x : m.y;
}

// Four dwords (8 BF16) -> two dwords (8 E4M3) with the block's inverse scale.
__device__ __forceinline__ v2i convert8(const uint32_t *d, float inv) {
    v2i out;
    int w0 = cvt2_e4m3<false>(bits_to_float(d[0] << 16) * inv,
                              bits_to_float(d[0] & 0xFFFF0000u) * inv, 0);
    w0 = cvt2_e4m3<true>(bits_to_float(d[1] << 16) * inv,
                         bits_to_float(d[1] & 0xFFFF0000u) * inv, w0);
    int w1 = cvt2_e4m3<false>(bits_to_float(d[2] << 16) * inv,
                              bits_to_float(d[2] & 0xFFFF0000u) * inv, 0);
    w1 = cvt2_e4m3<true>(bits_to_float(d[3] << 16) * inv,
                         bits_to_float(d[3] & 0xFFFF0000u) * inv, w1);
    out.x = w0;
    out.y = w1;
    return out;
}

// quad_perm DPP control [1,0,3,2]: swap the lanes of each pair
constexpr int kQuadSwap1 = 0xB1;

}  // namespace mx
