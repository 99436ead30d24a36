// Wavefront building blocks of the token-level kernels:
// reductions over aligned groups of lanes, vector loads of any alignment,
// order-preserving integer keys, and exponentials.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.hpp"

namespace mx {

// ---------------------------------------------------------------- lane groups

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t lane_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t lane_bits(uint32_t v) { return v; }
template <class T>
__device__ __forceinline__ T from_bits(uint32_t u);
template <>
__device__ __forceinline__ float from_bits<float>(uint32_t u) { return __uint_as_float(u); }
template <>
__device__ __forceinline__ uint32_t from_bits<uint32_t>(uint32_t u) { return u; }

struct OpMax {
    __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct OpMin {
    __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fminf(a, b); }
};
struct OpAdd {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// The value of the partner lane of butterfly step STEP (lane distance 2^STEP).
// Inside a row of 16 lanes the step is a lane permutation of the vector ALU:
// a swap of neighbours, a swap of pairs, then two mirrors, which stand for
// distance 4 and 8 because the lanes that the earlier steps joined already
// agree.  Steps 4 and 5 go through the LDS crossbar.
template <int STEP, class T>
__device__ __forceinline__ T partner(T v) {
    if constexpr (STEP == 0) return from_bits<T>(dpp_mov<0xB1>(lane_bits(v)));    // quad_perm 1,0,3,2
    if constexpr (STEP == 1) return from_bits<T>(dpp_mov<0x4E>(lane_bits(v)));    // quad_perm 2,3,0,1
    if constexpr (STEP == 2) return from_bits<T>(dpp_mov<0x141>(lane_bits(v)));   // row_half_mirror
    if constexpr (STEP == 3) return from_bits<T>(dpp_mov<0x140>(lane_bits(v)));   // row_mirror
    if constexpr (STEP >= 4) return from_bits<T>((uint32_t)__shfl_xor((int)lane_bits(v), 1 << STEP, 64));
}

// Reduction over aligned groups of W lanes (a power of two); every lane gets
// its group's result.  All 64 lanes have to take part.
template <int W, class T, class Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
    if constexpr (W >= 2) v = op(v, partner<0>(v));
    if constexpr (W >= 4) v = op(v, partner<1>(v));
    if constexpr (W >= 8) v = op(v, partner<2>(v));
    if constexpr (W >= 16) v = op(v, partner<3>(v));
    if constexpr (W >= 32) v = op(v, partner<4>(v));
    if constexpr (W >= 64) v = op(v, partner<5>(v));
    return v;
}

// LDS written by a lane, read by another of its wave
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------- vector access

// 16 bytes at any element-aligned address: gfx950's global loads and stores
// take unaligned addresses, so a row of odd length costs no scalar path.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
struct __attribute__((packed)) Bytes16 {
    v4u v;
};
template <class P>
__device__ __forceinline__ v4u load16(const P *p) {
    return reinterpret_cast<const Bytes16 *>(p)->v;
}
template <class P>
__device__ __forceinline__ void store16(P *p, v4u v) {
    reinterpret_cast<Bytes16 *>(p)->v = v;
}

// The same with ONCE for data that a pass reads or writes once and that is too
// large to stay in the last-level cache: nontemporal, so that it does not push
// through the caches.
constexpr int64_t kLastLevelBytes = 256 << 20;
template <class P>
struct Once16 {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Once16<uint16_t> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <bool ONCE, class P>
__device__ __forceinline__ v4u load16(const P *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const typename Once16<P>::type *>(p));
    else return load16(p);
}
template <bool ONCE, class P>
__device__ __forceinline__ void store16(P *p, v4u v) {
    if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<typename Once16<P>::type *>(p));
    else store16(p, v);
}

// Element types of the calls: fp32, or bf16 as its bit pattern.
template <class E>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;      // elements in 16 bytes
    __device__ static __forceinline__ float get(float v) { return v; }
    __device__ static __forceinline__ float put(float v) { return v; }
    __device__ static __forceinline__ void unpack(v4u r, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
    }
    __device__ static __forceinline__ v4u pack(const float *f) {
        return v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};
template <>
struct Elem<uint16_t> {
    static constexpr int kVec = 8;
    __device__ static __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static __forceinline__ uint16_t put(float v) { return (uint16_t)f32_to_bf16_rne(v); }
    __device__ static __forceinline__ void unpack(v4u r, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(r[i] << 16);
            f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
    __device__ static __forceinline__ v4u pack(const float *f) {
        return v4u{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
    }
};

// The first `count` of N values at p, the rest `pad`.  Loads without a branch:
// one each element would cost a round trip each.  p[0] is read whatever count is.
template <int N, class E>
__device__ __forceinline__ void load_head(const E *p, int count, float pad, float *x) {
    E r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = p[i < count ? i : 0];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < count ? Elem<E>::get(r[i]) : pad;
}

// ---------------------------------------------------------------- keys

// Unsigned integers in the order of the floats (-Inf lowest; a NaN above
// +Inf or below -Inf by its sign, so every bit pattern has a place).
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ uint64_t order_key(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// ---------------------------------------------------------------- exponentials

constexpr float kLog2E = 1.44269504088896f;
constexpr float kLog2ELow = 1.92596302e-8f;   // log2(e) - (float)log2(e)
constexpr float kLn2 = 0.693147180559945f;

// e^d for d <= 0 (or NaN) at about fp32's last place: the hardware's 2^x on
// the rounded product d * log2(e), and the product's rounding error put back
// to first order.  Without that the error grows as |d| * 2^-24.
__device__ __forceinline__ float exp_neg(float d) {
    d = d < -200.0f ? -200.0f : d;            // 0 either way; keeps the residue finite, passes NaN
    const float h = d * kLog2E;
    const float r = __builtin_fmaf(d, kLog2ELow, __builtin_fmaf(d, kLog2E, -h));
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, r * kLn2, e);
}

// 1 / (1 + e^-x), from e^-|x| so that neither side overflows
__device__ __forceinline__ float sigmoid(float x) {
    const float e = exp_neg(-__builtin_fabsf(x));
    return (x < 0.0f ? e : 1.0f) / (1.0f + e);
}

}  // namespace mx
