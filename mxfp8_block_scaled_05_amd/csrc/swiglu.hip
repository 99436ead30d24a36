// The gated activation h = silu(gate) * up, with gate and up kept as MXFP8 for
// the backward pass, and its gradient from that checkpoint.
//
// Both directions stream: a lane owns 16 columns of gate and the same 16 of up
// (a half block of each, so a block's scale needs one swap within a lane pair,
// as in the axis-1 quantizer), and everything that the values lead to is
// computed while they are in registers.
#include "mx_convert.hpp"
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;
constexpr int kPerCu = 8;           // blocks of the walk for every compute unit

// s = 1 / (1 + e^-g) and 1 - s, both from e^-|g|, so that neither side
// overflows or cancels.  |g| log2(e) is rounded once, which costs |g| 2^-24
// of the result: below 2^-17 wherever s is above fp32's smallest number.
struct Gate {
    float s, rest;
};
__device__ __forceinline__ Gate gate_of(float g) {
    const float t = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * kLog2E);
    const float r = __builtin_amdgcn_rcpf(1.0f + t), low = t * r;
    return g < 0.0f ? Gate{low, r} : Gate{r, low};
}

__device__ __forceinline__ void unpack16(const v4u *r, float *f) {
    Elem<uint16_t>::unpack(r[0], f);
    Elem<uint16_t>::unpack(r[1], f + 8);
}

// a half block's 16 values to codes; the lane pair shares the block's scale code
__device__ __forceinline__ uint32_t block_code(const v4u *r) {
    uint32_t d[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
    uint32_t m = max_mag(d, 8);
    const uint32_t other = dpp_mov<kQuadSwap1>(m);
    return scale_code_from_amax_bits(m > other ? m : other);
}
__device__ __forceinline__ v4i codes16(const v4u *r, uint32_t code) {
    const uint32_t lo[4] = {r[0].x, r[0].y, r[0].z, r[0].w}, hi[4] = {r[1].x, r[1].y, r[1].z, r[1].w};
    const float inv = inv_scale_from_code(code);
    const v2i a = convert8(lo, inv), b = convert8(hi, inv);
    return code == 255u ? v4i{0x7F7F7F7F, 0x7F7F7F7F, 0x7F7F7F7F, 0x7F7F7F7F} : v4i{a.x, a.y, b.x, b.y};
}

enum class H { kBf16, kCanonical, kPacked };

// What a step of 64 lanes covers.  Rows in order: 64 half blocks of the flat
// [T][I / 16] array.  Packed: 8 rows x 128 columns of one tile of the layout,
// over every row of every panel, so that a step's codes are 1 KB of it.
template <H FORM>
struct Place {
    int64_t row;
    int col;
    bool real;
};
template <H FORM>
__device__ __forceinline__ Place<FORM> place_of(const SwigluArgs &a, uint32_t step, int lane, uint32_t halves) {
    if constexpr (FORM == H::kPacked) {
        const uint32_t KS = (uint32_t)((a.I + 127) >> 7);
        const uint32_t band = step / KS, ks = step - band * KS;
        const int64_t row = (int64_t)band * 8 + (lane >> 3);
        const int col = (int)ks * 128 + (lane & 7) * 16;
        return {row, col, row < a.T && col < a.I};
    } else {
        const uint32_t at = step * 64 + lane, per = (uint32_t)a.I >> 4;
        const uint32_t row = at / per;
        return {(int64_t)row, (int)((at - row * per) << 4), at < halves};
    }
}

template <H FORM>
__global__ __launch_bounds__(kBlock) void swiglu_kernel(const SwigluArgs a, uint32_t steps, uint32_t halves) {
    const int lane = threadIdx.x & 63;
    const uint32_t waves = gridDim.x * (kBlock / 64);
    for (uint32_t step = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); step < steps; step += waves) {
        const Place<FORM> p = place_of<FORM>(a, step, lane, halves);
        v4u g[2] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}}, u[2] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}};
        if (p.real) {
            const v4u *at = reinterpret_cast<const v4u *>(a.x + p.row * a.ld + p.col);
            const v4u *up = reinterpret_cast<const v4u *>(a.x + p.row * a.ld + a.I + p.col);
            g[0] = at[0], g[1] = at[1], u[0] = up[0], u[1] = up[1];
        }
        if (a.q) {                                       // uniform
            const uint32_t cg = block_code(g), cu = block_code(u);
            if (p.real) {
                uint8_t *q = a.q + p.row * 2 * a.I + p.col;
                *reinterpret_cast<v4i *>(q) = codes16(g, cg);
                *reinterpret_cast<v4i *>(q + a.I) = codes16(u, cu);
                if (!(lane & 1)) {
                    uint8_t *s = a.s + p.row * (a.I >> 4) + (p.col >> 5);
                    s[0] = (uint8_t)cg;
                    s[a.I >> 5] = (uint8_t)cu;
                }
            }
        }
        float fg[16], fu[16];
        unpack16(g, fg), unpack16(u, fu);
#pragma unroll
        for (int i = 0; i < 16; ++i) fg[i] = fg[i] * gate_of(fg[i]).s * fu[i];
        const v4u h[2] = {Elem<uint16_t>::pack(fg), Elem<uint16_t>::pack(fg + 8)};
        if constexpr (FORM == H::kBf16) {
            if (p.real) {
                v4u *out = reinterpret_cast<v4u *>(a.h + p.row * a.I + p.col);
                out[0] = h[0], out[1] = h[1];
            }
        } else {
            uint32_t code = block_code(h);
            if constexpr (FORM == H::kCanonical) {
                if (p.real) {
                    *reinterpret_cast<v4i *>(a.hq + p.row * a.I + p.col) = codes16(h, code);
                    if (!(lane & 1)) a.hs[p.row * (a.I >> 5) + (p.col >> 5)] = (uint8_t)code;
                }
            } else {
                const v4i q = codes16(h, code);          // zeros where there is no value
                if (!p.real) code = 127u;                // the layout's padding scale
                const int64_t tile = (p.row >> 8) * ((a.I + 127) >> 7) + (p.col >> 7);
                const int r = (int)(p.row & 255), c = (p.col & 127) >> 4;
                *reinterpret_cast<v4i *>(a.hq + tile * kTileBytes + r * 128 + ((c ^ (int)swz((uint32_t)r)) << 4)) = q;
                if (!(lane & 1)) a.hs[tile * kScaleStepBytes + (r >> 4) * 64 + (c >> 1) * 16 + (r & 15)] = (uint8_t)code;
            }
        }
    }
}

// 2^(code - 127), NaN for 255
__device__ __forceinline__ float scale_value(uint32_t code) {
    return bits_to_float(code == 0u ? 0x00400000u : code == 255u ? 0x7FC00000u : code << 23);
}
__device__ __forceinline__ void values16(v4i q, float scale, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
        f[4 * i] = lo.x * scale, f[4 * i + 1] = lo.y * scale;
        f[4 * i + 2] = hi.x * scale, f[4 * i + 3] = hi.y * scale;
    }
}

__global__ __launch_bounds__(kBlock) void swiglu_backward_kernel(const SwigluArgs a, uint32_t steps, uint32_t halves) {
    const int lane = threadIdx.x & 63;
    const uint32_t waves = gridDim.x * (kBlock / 64);
    for (uint32_t step = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); step < steps; step += waves) {
        const Place<H::kBf16> p = place_of<H::kBf16>(a, step, lane, halves);
        if (!p.real) continue;
        const v4u *at = reinterpret_cast<const v4u *>(a.x + p.row * a.ld + p.col);
        const v4u d[2] = {at[0], at[1]};
        const uint8_t *q = a.q + p.row * 2 * a.I + p.col, *s = a.s + p.row * (a.I >> 4) + (p.col >> 5);
        const v4i qg = *reinterpret_cast<const v4i *>(q), qu = *reinterpret_cast<const v4i *>(q + a.I);
        const float sg = scale_value(s[0]), su = scale_value(s[a.I >> 5]);
        float g[16], u[16], dh[16];
        values16(qg, sg, g), values16(qu, su, u), unpack16(d, dh);
        float dg[16], du[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const Gate t = gate_of(g[i]);
            const float silu = g[i] * t.s;
            du[i] = dh[i] * silu;
            dg[i] = dh[i] * u[i] * __builtin_fmaf(silu, t.rest, t.s);      // s + g s (1 - s)
            g[i] = silu * u[i];
        }
        v4u *out = reinterpret_cast<v4u *>(a.dx + p.row * 2 * a.I + p.col);
        out[0] = Elem<uint16_t>::pack(dg), out[1] = Elem<uint16_t>::pack(dg + 8);
        out = reinterpret_cast<v4u *>(a.dx + p.row * 2 * a.I + a.I + p.col);
        out[0] = Elem<uint16_t>::pack(du), out[1] = Elem<uint16_t>::pack(du + 8);
        if (a.h) {
            out = reinterpret_cast<v4u *>(a.h + p.row * a.I + p.col);
            out[0] = Elem<uint16_t>::pack(g), out[1] = Elem<uint16_t>::pack(g + 8);
        }
    }
}

unsigned grid_of(uint32_t steps) {
    const int64_t blocks = ceil_div(steps, kBlock / 64), most = (int64_t)device_cu_count() * kPerCu;
    return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs &a, bool h_packed, hipStream_t stream) {
    const uint32_t halves = (uint32_t)(a.T * (a.I / 16));
    if (a.hq && h_packed) {
        const uint32_t steps = (uint32_t)(packed_panels(a.T) * 32 * packed_ksteps(a.I));
        swiglu_kernel<H::kPacked><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, halves);
        return hipGetLastError();
    }
    const uint32_t steps = (uint32_t)ceil_div(halves, 64);
    if (a.hq) swiglu_kernel<H::kCanonical><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, halves);
    else swiglu_kernel<H::kBf16><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, halves);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const SwigluArgs &a, hipStream_t stream) {
    const uint32_t halves = (uint32_t)(a.T * (a.I / 16)), steps = (uint32_t)ceil_div(halves, 64);
    swiglu_backward_kernel<<<grid_of(steps), kBlock, 0, stream>>>(a, steps, halves);
    return hipGetLastError();
}

}  // namespace mx
