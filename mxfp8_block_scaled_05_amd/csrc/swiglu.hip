// The gated activation h = silu(gate) * up, with gate and up kept as MXFP8 for
// the backward pass, and its gradient from that checkpoint.
//
// Both directions stream, and HBM bounds them: 8192 x 12288 (714 MB with the
// checkpoint and codes of h) in 116 us (its vector arithmetic takes as long), the
// gradient of 4095 x 12288 (507 MB) in 82 us, 6.2 TB/s both.  The forward pass
// into the packed layout takes 121 us; without a checkpoint 83, packed or not;
// with h in bf16 130, and 94 without a checkpoint.  A lane owns 8 columns of gate
// and the same 8 of up, so that a wave's accesses are whole runs of 1 KB (512 B of
// codes), and four lanes share a block's scale; with 16 columns a lane, two
// accesses of every second 16 bytes, the same take 142 and 107.  Everything that
// the values lead to is computed while they are in registers, and stored together
// at the end (codes of gate and up stored before h is known: 121).
#include "mx_convert.hpp"
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;
// Blocks for every compute unit, at most: a wave takes one step or a few, and
// the next block's loads overlap its stores (8 blocks that walk: 134 us and 98).
constexpr int kPerCu = 128;

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

// the block's scale code, from the four lanes that hold its values
__device__ __forceinline__ uint32_t block_code(v4u r) {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
    const uint32_t m = group_reduce<4>(max_mag(d, 4), OpMax());
    return scale_code_from_amax_bits(m);
}
__device__ __forceinline__ v2i codes8(v4u r, uint32_t code) {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
    const v2i q = convert8(d, inv_scale_from_code(code));
    return code == 255u ? v2i{0x7F7F7F7F, 0x7F7F7F7F} : q;
}

// 8 bytes of codes, ONCE as load16's and store16's
template <bool ONCE>
__device__ __forceinline__ v2i load8(const uint8_t *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const v2i *>(p));
    else return *reinterpret_cast<const v2i *>(p);
}
template <bool ONCE>
__device__ __forceinline__ void store8(uint8_t *p, v2i v) {
    if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<v2i *>(p));
    else *reinterpret_cast<v2i *>(p) = v;
}

enum class H { kBf16, kCanonical, kPacked };

// What a step of 64 lanes covers.  Rows in order: 64 runs of 8 columns of the
// flat [T][I / 8] array.  Packed: 4 rows x 128 columns of one tile of the
// layout, over every row of every panel, so that a step's codes are 512 B of it.
struct Place {
    int64_t row;
    int col;
    bool real;
};
template <H FORM>
__device__ __forceinline__ Place place_of(const SwigluArgs &a, uint32_t step, int lane, uint32_t runs) {
    if constexpr (FORM == H::kPacked) {
        const uint32_t KS = (uint32_t)((a.I + 127) >> 7);
        const uint32_t band = step / KS, ks = step - band * KS;
        const int64_t row = (int64_t)band * 4 + (lane >> 4);
        const int col = (int)ks * 128 + (lane & 15) * 8;
        return {row, col, row < a.T && col < a.I};
    } else {
        const uint32_t at = step * 64 + lane, per = (uint32_t)a.I >> 3;
        const uint32_t row = at / per;
        return {(int64_t)row, (int)((at - row * per) << 3), at < runs};
    }
}

template <H FORM, bool ONCE>
__global__ __launch_bounds__(kBlock) void swiglu_kernel(const SwigluArgs a, uint32_t steps, uint32_t runs) {
    const int lane = threadIdx.x & 63;
    const uint32_t waves = gridDim.x * (kBlock / 64);
    for (uint32_t step = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); step < steps; step += waves) {
        const Place p = place_of<FORM>(a, step, lane, runs);
        v4u g = v4u{0, 0, 0, 0}, u = g;
        if (p.real) {
            const uint16_t *x = a.x + p.row * a.ld + p.col;
            g = load16<ONCE>(x), u = load16<ONCE>(x + a.I);
        }
        float fg[8], fu[8];
        Elem<uint16_t>::unpack(g, fg), Elem<uint16_t>::unpack(u, fu);
#pragma unroll
        for (int i = 0; i < 8; ++i) fg[i] = fg[i] * gate_of(fg[i]).s * fu[i];
        const v4u h = Elem<uint16_t>::pack(fg);
        if (a.q) {                                       // uniform
            const uint32_t cg = block_code(g), cu = block_code(u);
            if (p.real) {
                uint8_t *q = a.q + p.row * 2 * a.I + p.col;
                store8<ONCE>(q, codes8(g, cg));
                store8<ONCE>(q + a.I, codes8(u, cu));
                if (!(lane & 3)) {
                    uint8_t *s = a.s + p.row * (a.I >> 4) + (p.col >> 5);
                    s[0] = (uint8_t)cg;
                    s[a.I >> 5] = (uint8_t)cu;
                }
            }
        }
        if constexpr (FORM == H::kBf16) {
            if (p.real) store16<ONCE>(a.h + p.row * a.I + p.col, h);
        } else {
            uint32_t code = block_code(h);
            if constexpr (FORM == H::kCanonical) {
                if (p.real) {
                    store8<ONCE>(a.hq + p.row * a.I + p.col, codes8(h, code));
                    if (!(lane & 3)) a.hs[p.row * (a.I >> 5) + (p.col >> 5)] = (uint8_t)code;
                }
            } else {
                const v2i q = codes8(h, code);           // zeros where there is no value
                if (!p.real) code = 127u;                // the layout's padding scale
                const int64_t tile = (p.row >> 8) * ((a.I + 127) >> 7) + (p.col >> 7);
                const int r = (int)(p.row & 255), c = (p.col & 127) >> 4;
                store8<ONCE>(a.hq + tile * kTileBytes + r * 128 + ((c ^ (int)swz((uint32_t)r)) << 4) + (p.col & 8), q);
                if (!(lane & 3)) a.hs[tile * kScaleStepBytes + (r >> 4) * 64 + (c >> 1) * 16 + (r & 15)] = (uint8_t)code;
            }
        }
    }
}

// 2^(code - 127), NaN for 255
__device__ __forceinline__ float scale_value(uint32_t code) {
    return bits_to_float(code == 0u ? 0x00400000u : code == 255u ? 0x7FC00000u : code << 23);
}
__device__ __forceinline__ void values8(v2i q, float scale, float *f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
        f[4 * i] = lo.x * scale, f[4 * i + 1] = lo.y * scale;
        f[4 * i + 2] = hi.x * scale, f[4 * i + 3] = hi.y * scale;
    }
}

template <bool ONCE>
__global__ __launch_bounds__(kBlock) void swiglu_backward_kernel(const SwigluArgs a, uint32_t steps, uint32_t runs) {
    const uint32_t waves = gridDim.x * (kBlock / 64);
    for (uint32_t step = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); step < steps; step += waves) {
        const Place p = place_of<H::kBf16>(a, step, threadIdx.x & 63, runs);
        if (!p.real) continue;
        const v4u d = load16<ONCE>(a.x + p.row * a.ld + p.col);
        const uint8_t *q = a.q + p.row * 2 * a.I + p.col, *s = a.s + p.row * (a.I >> 4) + (p.col >> 5);
        const v2i qg = load8<ONCE>(q), qu = load8<ONCE>(q + a.I);
        float g[8], u[8], dh[8], dg[8], du[8];
        values8(qg, scale_value(s[0]), g), values8(qu, scale_value(s[a.I >> 5]), u), Elem<uint16_t>::unpack(d, dh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Gate t = gate_of(g[i]);
            const float silu = g[i] * t.s;
            du[i] = dh[i] * silu;
            dg[i] = dh[i] * u[i] * __builtin_fmaf(silu, t.rest, t.s);          // s + g s (1 - s)
            g[i] = silu * u[i];
        }
        uint16_t *out = a.dx + p.row * 2 * a.I + p.col;
        store16<ONCE>(out, Elem<uint16_t>::pack(dg));
        store16<ONCE>(out + a.I, Elem<uint16_t>::pack(du));
        if (a.h) store16<ONCE>(a.h + p.row * a.I + p.col, Elem<uint16_t>::pack(g));
    }
}

unsigned grid_of(uint32_t steps) {
    const int64_t blocks = ceil_div(steps, kBlock / 64), most = (int64_t)device_cu_count() * kPerCu;
    return (unsigned)(blocks < most ? blocks : most);
}

// Past the caches where the pass moves more than the last level holds: what it
// wrote first is not there any more when the next call comes (8192 x 12288 126 us
// through the caches, the gradient of 4095 x 12288 88).
bool moves_more(int64_t bytes) { return bytes > kLastLevelBytes; }

template <H FORM>
hipError_t start(const SwigluArgs &a, uint32_t steps, uint32_t runs, bool once, hipStream_t stream) {
    if (once) swiglu_kernel<FORM, true><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, runs);
    else swiglu_kernel<FORM, false><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, runs);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs &a, bool h_packed, hipStream_t stream) {
    const int64_t n = a.T * a.I;
    const uint32_t runs = (uint32_t)(n / 8), steps = (uint32_t)ceil_div(n, 512);
    const bool once = moves_more(n * (4 + (a.q ? 2 : 0) + (a.h ? 2 : 1)));
    if (a.h) return start<H::kBf16>(a, steps, runs, once, stream);
    if (!h_packed) return start<H::kCanonical>(a, steps, runs, once, stream);
    return start<H::kPacked>(a, (uint32_t)(packed_panels(a.T) * 64 * packed_ksteps(a.I)), runs, once, stream);
}

hipError_t launch_swiglu_backward(const SwigluArgs &a, hipStream_t stream) {
    const int64_t n = a.T * a.I;
    const uint32_t runs = (uint32_t)(n / 8), steps = (uint32_t)ceil_div(n, 512);
    if (moves_more(n * (a.h ? 10 : 8))) swiglu_backward_kernel<true><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, runs);
    else swiglu_backward_kernel<false><<<grid_of(steps), kBlock, 0, stream>>>(a, steps, runs);
    return hipGetLastError();
}

}  // namespace mx
