// Low-rank adapters of many requests beside a shared projection: y += s B (A x)
// for rows sorted by adapter, and the gradients of x, A and B.
//
// A group's rows start at a multiple of 32, so every block of 32 sorted rows
// has one adapter and its products run on the matrix unit.  The rank is small:
// every product reads or writes one wide matrix once and is bound by that, so
// operands go from global memory straight into matrix fragments (the weights'
// and hidden rows' fragments come from the caches) and LDS only joins waves.
//
//   shrink   P = X A^T          partial sums over slices of the wide axis
//   expand   Y += (s P) B^T     sums the partials, keeps P
//   outer    W = (s P)^T X      sums over rows, per adapter
// Forward: shrink (x, A), expand (y, B).  Backward, with the transposed weights:
// shrink (d_y, B^T), expand (d_x, A^T), outer twice (d_a: S and x; d_b: hidden
// and d_y).
//
// P is held in fp32.  Where it is an operand of the matrix unit it enters as
// two bf16 numbers, hi + lo, which keep 16 bits of it (2^-16 of the value lost;
// a single one would lose 2^-8, more than bf16 inputs allow the fp32 gradients
// of the weights).  The second product costs matrix time that is idle anyway.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kRows = 32;           // sorted rows that share an adapter
constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Two values as hi + lo, each pair of bf16 in a word.  What the rounding to bf16
// takes to infinity, or was infinite, has no rest.
__device__ __forceinline__ float rest_of(float v, float hi) {
    const float d = v - hi;
    return d == d ? d : 0.0f;
}
__device__ __forceinline__ void split2(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    hi = bf16x2_rne(v0, v1);
    lo = bf16x2_rne(rest_of(v0, __uint_as_float(hi << 16)), rest_of(v1, __uint_as_float(hi & 0xFFFF0000u)));
}

// The number of offsets[0..E] that are at most row, less one: the group that
// the row lies in (-1 or E: none).  All lanes of the wave take part.
__device__ __forceinline__ int adapter_of(const int32_t *offsets, int E, int row, int lane) {
    int n = 0;
    for (int i = 0; i <= E; i += 64) {
        const int at = i + lane;
        const int v = offsets[at <= E ? at : E];
        n += __builtin_popcountll(__ballot(at <= E && v <= row));
    }
    return n - 1;
}

// The token of a sorted row, -1 for padding
__device__ __forceinline__ int token_of(const int64_t *row_token, int64_t row, int64_t T) {
    const int64_t t = row_token[row];
    return t >= 0 && t < T ? (int)t : -1;
}

// ---------------------------------------------------------------- shrink

// One block: 32 sorted rows, a slice of the wide axis, all ranks.  Its waves
// take chunks of 128 columns in turn.  RT: tiles of 16 ranks.
template <int RT>
__global__ __launch_bounds__(kBlock) void lora_shrink_kernel(const LoraShrink a) {
    __shared__ v4f red[kWaves][kRows][RT * 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, kg = lane >> 4;
    const int rb = blockIdx.x / a.splits, split = blockIdx.x - rb * a.splits;
    const int e = adapter_of(a.offsets, a.E, rb * kRows, lane);
    if (e < 0 || e >= a.E) return;                       // the whole block
    const uint16_t *x[2];
    bool real[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int token = token_of(a.row_token, (int64_t)rb * kRows + t * 16 + m, a.T);
        real[t] = token >= 0;
        x[t] = a.x + (real[t] ? token : 0) * a.ld;
    }
    const bool second = __ballot(real[1]) != 0;
    const uint16_t *w[RT];
    bool rank[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        rank[j] = j * 16 + m < a.r;
        w[j] = a.w + ((int64_t)e * a.r + (rank[j] ? j * 16 + m : 0)) * a.K;
    }
    v4f acc[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[t][j] = v4f{0, 0, 0, 0};
    const v4u zero = {0, 0, 0, 0};
    const int k1 = min(a.K, (split + 1) * a.slice);
    for (int k0 = split * a.slice + wave * 128; k0 < k1; k0 += kWaves * 128) {
        v4u xf[4][2], wf[4][RT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = k0 + s * 32 + kg * 8;
            const bool in = k < k1;
            const int at = in ? k : 0;
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t == 0 || second) {
                    const v4u v = *reinterpret_cast<const v4u *>(x[t] + at);
                    xf[s][t] = in && real[t] ? v : zero;
                }
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const v4u v = *reinterpret_cast<const v4u *>(w[j] + at);
                wf[s][j] = in && rank[j] ? v : zero;
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t == 0 || second) {
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[t][j] = mfma(wf[s][j], xf[s][t], acc[t][j]);
                }
    }
    // a lane holds four ranks, 4 kg.., of row m
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < RT; ++j) red[wave][t * 16 + m][j * 4 + kg] = acc[t][j];
    __syncthreads();
    float *out = a.part + ((int64_t)split * a.rows + (int64_t)rb * kRows) * a.r;
    for (int i = threadIdx.x; i < kRows * RT * 4; i += kBlock) {
        const int row = i / (RT * 4), q = i - row * (RT * 4);
        if (q * 4 >= a.r) continue;
        v4f v = red[0][row][q];
#pragma unroll
        for (int n = 1; n < kWaves; ++n) v += red[n][row][q];
        *reinterpret_cast<v4f *>(out + (int64_t)row * a.r + q * 4) = v;
    }
}

// ---------------------------------------------------------------- expand

// 16 consecutive values of a row of y, those below `left` columns (a multiple of 8)
template <class Y>
struct Run16;
template <>
struct Run16<uint16_t> {
    v4u r[2];
    __device__ __forceinline__ void load(const uint16_t *p, int left) {
        if (left > 0) r[0] = *reinterpret_cast<const v4u *>(p);
        if (left > 8) r[1] = *reinterpret_cast<const v4u *>(p + 8);
    }
    __device__ __forceinline__ void add_store(uint16_t *p, int left, const v4f *d) {
        float f[16];
        Elem<uint16_t>::unpack(r[0], f), Elem<uint16_t>::unpack(r[1], f + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] += d[i >> 2][i & 3];
        if (left > 0) *reinterpret_cast<v4u *>(p) = Elem<uint16_t>::pack(f);
        if (left > 8) *reinterpret_cast<v4u *>(p + 8) = Elem<uint16_t>::pack(f + 8);
    }
};
template <>
struct Run16<float> {
    v4f r[4];
    __device__ __forceinline__ void load(const float *p, int left) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (left > i * 4) r[i] = *reinterpret_cast<const v4f *>(p + i * 4);
    }
    __device__ __forceinline__ void add_store(float *p, int left, const v4f *d) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (left > i * 4) *reinterpret_cast<v4f *>(p + i * 4) = r[i] + d[i];
    }
};

// One block: RB groups of 32 sorted rows x 256 columns, a wave 64 of them.  The
// products are taken as B P^T, with the rows of B that a tile of 16 takes chosen
// so that a lane ends up with 16 consecutive columns of one row of y.
// KT: steps of 32 ranks.
template <class Y, int KT, int RB>
__global__ __launch_bounds__(kBlock) void lora_expand_kernel(const LoraExpand a) {
    __shared__ v4u frag[RB * 2][KT][2][64];              // P of each 16 rows as the matrix unit takes it: hi, lo
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, kg = lane >> 4;
    const int group = blockIdx.x / a.tiles, tile = blockIdx.x - group * a.tiles;
    const int rb0 = group * RB;
    const int blocks = (int)(a.rows / kRows);
    int e[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        e[i] = rb0 + i < blocks ? adapter_of(a.offsets, a.E, (rb0 + i) * kRows, lane) : -1;
        if (e[i] >= a.E) e[i] = -1;
    }
    for (int i = threadIdx.x; i < RB * 2 * KT * 64; i += kBlock) {
        const int l = i & 63, kt = (i >> 6) % KT, mt = (i >> 6) / KT;
        const int ee = RB == 1 ? e[0] : mt < 2 ? e[0] : mt < 4 ? e[RB > 1 ? 1 : 0] : mt < 6 ? e[RB > 2 ? 2 : 0] : e[RB > 3 ? 3 : 0];
        const int64_t row = (int64_t)rb0 * kRows + mt * 16 + (l & 15);
        const int j = kt * 32 + (l >> 4) * 8;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const bool in = j < a.r && row < a.rows;
        if (in && ee >= 0) {
            const float *p = a.part + row * a.r + j;
            for (int s = 0; s < a.splits; ++s, p += a.rows * a.r) {
                const v4f lo = *reinterpret_cast<const v4f *>(p), hi = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += lo[q], v[4 + q] += hi[q];
            }
        }
        if (a.hidden && tile == 0 && in) {
            float *h = a.hidden + row * a.r + j;
            *reinterpret_cast<v4f *>(h) = v4f{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<v4f *>(h + 4) = v4f{v[4], v[5], v[6], v[7]};
        }
        const float scale = a.scales && ee >= 0 ? a.scales[ee] : 1.0f;
        v4u hi, lo;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t h, l2;
            split2(v[2 * q] * scale, v[2 * q + 1] * scale, h, l2);
            hi[q] = h, lo[q] = l2;
        }
        frag[mt][kt][0][l] = hi;
        frag[mt][kt][1][l] = lo;
    }
    __syncthreads();
    const int c0 = tile * 256 + wave * 64;
    if (c0 >= a.N) return;
    const int left = a.N - c0 - kg * 16;                 // columns from this lane's first on
    v4u b[4][KT];
    int held = -1;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        if (e[i] < 0) continue;
        if (e[i] != held) {
            held = e[i];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = c0 + (m >> 2) * 16 + q * 4 + (m & 3);
                const bool in = n < a.N;
                const uint16_t *row = a.w + ((int64_t)held * a.N + (in ? n : 0)) * a.r;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const int j = kt * 32 + kg * 8;
                    const v4u v = *reinterpret_cast<const v4u *>(row + (j < a.r ? j : 0));
                    b[q][kt] = in && j < a.r ? v : v4u{0, 0, 0, 0};
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int token = token_of(a.row_token, (int64_t)(rb0 + i) * kRows + t * 16 + m, a.T);
            if (__ballot(token >= 0) == 0) continue;
            Y *y = static_cast<Y *>(a.y) + (token < 0 ? 0 : token) * a.ld + c0 + kg * 16;
            const int take = token < 0 ? 0 : left;
            Run16<Y> run{};
            run.load(y, take);
            v4f d[4] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const v4u hi = frag[i * 2 + t][kt][0][lane], lo = frag[i * 2 + t][kt][1][lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) d[q] = mfma(b[q][kt], lo, d[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) d[q] = mfma(b[q][kt], hi, d[q]);
            }
            run.add_store(y, take, d);
        }
    }
}

// ---------------------------------------------------------------- transposed weights

// [E][P][Q] -> [E][Q][P], 64 x 64 tiles, P and Q multiples of 8
__global__ __launch_bounds__(kBlock) void lora_transpose_kernel(const LoraTranspose a) {
    __shared__ uint16_t t[64][72];
    const LoraTranspose::Job &job = a.job[blockIdx.y];
    const int across = (job.Q + 63) / 64, down = (job.P + 63) / 64;
    for (int64_t at = blockIdx.x; at < (int64_t)a.E * across * down; at += gridDim.x) {
        const int64_t e = at / (across * down);
        const int in = (int)(at - e * across * down);
        const int p0 = in / across * 64, q0 = in % across * 64;
        const uint16_t *from = job.from + e * job.P * job.Q;
        uint16_t *to = job.to + e * job.P * job.Q;
        for (int i = threadIdx.x; i < 512; i += kBlock) {
            const int p = i >> 3, q = (i & 7) * 8;
            if (p0 + p < job.P && q0 + q < job.Q)
                *reinterpret_cast<v4u *>(&t[p][q]) = *reinterpret_cast<const v4u *>(from + (int64_t)(p0 + p) * job.Q + q0 + q);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 512; i += kBlock) {
            const int q = i >> 3, p = (i & 7) * 8;
            if (p0 + p < job.P && q0 + q < job.Q) {
                v4u v;
#pragma unroll
                for (int n = 0; n < 4; ++n) v[n] = t[p + 2 * n][q] | ((uint32_t)t[p + 2 * n + 1][q] << 16);
                *reinterpret_cast<v4u *>(to + (int64_t)(q0 + q) * job.P + p0 + p) = v;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- outer products

// An adapter's rows are cut into items of `chunk`; one without rows has one
// empty item (its gradient is zeros).  Items of an adapter with several write
// partial sums into slots.
struct Item {
    int e, row0, row1;              // e < 0: there is no such item
    int slot;                       // -1: straight into the result
};
struct Scan {
    int items, slots, many;         // of the adapters before this lane's
    int m;                          // items of this lane's
};
__device__ __forceinline__ int lanes_before(int v, int lane) {
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64);
        s += lane >= d ? o : 0;
    }
    return s - v;
}
// adapters e0 + lane, with the totals so far in `before`
__device__ __forceinline__ Scan scan_adapters(const LoraOuter &a, int e0, int lane, const Scan &before, int &lo, int &hi) {
    const int e = e0 + lane, rows = (int)a.rows;
    lo = hi = 0;
    int m = 0;
    if (e < a.E) {
        lo = min(max(a.offsets[e], 0), rows);
        hi = max(min(max(a.offsets[e + 1], 0), rows), lo);
        lo &= ~(kRows - 1), hi &= ~(kRows - 1);          // a malformed table's rows stay whole blocks
        m = hi > lo ? (hi - lo + a.chunk - 1) / a.chunk : 1;
    }
    return Scan{before.items + lanes_before(m, lane), before.slots + lanes_before(m > 1 ? m : 0, lane),
                before.many + lanes_before(m > 1 ? 1 : 0, lane), m};
}
__device__ __forceinline__ Scan totals(const Scan &s) {
    return Scan{__shfl(s.items + s.m, 63, 64), __shfl(s.slots + (s.m > 1 ? s.m : 0), 63, 64),
                __shfl(s.many + (s.m > 1 ? 1 : 0), 63, 64), 0};
}
__device__ __forceinline__ Item item_of(const LoraOuter &a, int item, int lane) {
    Scan before{0, 0, 0, 0};
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        int lo, hi;
        const Scan s = scan_adapters(a, e0, lane, before, lo, hi);
        const uint64_t mine = __ballot(item >= s.items && item < s.items + s.m);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            const int part = item - __shfl(s.items, l, 64), m = __shfl(s.m, l, 64);
            lo = __shfl(lo, l, 64), hi = __shfl(hi, l, 64);
            const int slot = __shfl(s.slots, l, 64) + part;
            const int row0 = lo + part * a.chunk;
            return {e0 + l, row0, min(hi, row0 + a.chunk), m > 1 ? slot : -1};
        }
        before = totals(s);
    }
    return {-1, 0, 0, -1};
}

// The wide operand's 8 columns of 8 rows a lane, as fragments: f[c] holds
// column c of the eight rows (tokens), zeros for rows without one.
// The columns at `col` exist where `in`.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
struct WideBf16 {
    v4u r[8];
    __device__ __forceinline__ void load(const LoraWide &w, const int *token, int col, bool in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool real = token[i] >= 0 && in;
            const v4u v = *reinterpret_cast<const v4u *>(static_cast<const uint16_t *>(w.x) + (real ? token[i] * w.ld + col : 0));
            r[i] = real ? v : v4u{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ v4u column(int c) const {
        v4u f;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            f[d] = c & 1 ? high_halves(r[2 * d][c >> 1], r[2 * d + 1][c >> 1]) : low_halves(r[2 * d][c >> 1], r[2 * d + 1][c >> 1]);
        return f;
    }
};
// An MXFP8 grid, canonical or packed.  A value is 4 bits of E4M3 times a power
// of two: its upper 16 bits as an fp32 are the bf16 (below 2^-133 what is left
// of it).
template <bool PACKED>
struct WideGrid {
    v2i q[8];
    float scale[8];
    __device__ __forceinline__ void load(const LoraWide &w, const int *token, int col, bool in) {
        const uint8_t *x = static_cast<const uint8_t *>(w.x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool real = token[i] >= 0 && in;
            const int t = real ? token[i] : 0, c = real ? col : 0;
            int64_t at, sat;
            if constexpr (PACKED) {
                const int64_t tile = (int64_t)(t >> 8) * w.ksteps + (c >> 7);
                const int row = t & 255, chunk = (c & 127) >> 4;
                at = tile * kTileBytes + row * 128 + ((chunk ^ (int)swz((uint32_t)row)) << 4) + (c & 8);
                sat = tile * kScaleStepBytes + (row >> 4) * 64 + (chunk >> 1) * 16 + (row & 15);
            } else {
                at = t * w.ld + c;
                sat = t * (w.ld >> 5) + (c >> 5);
            }
            const v2i v = *reinterpret_cast<const v2i *>(x + at);
            const uint32_t code = w.s[sat];
            q[i] = real ? v : v2i{0, 0};
            scale[i] = bits_to_float(code == 0u ? 0x00400000u : code == 255u ? 0x7FC00000u : code << 23);
            if (!real) scale[i] = 0.0f;
        }
    }
    __device__ __forceinline__ float value(int i, int c) const {
        const int word = c & 4 ? q[i].y : q[i].x;
        const v2f v = c & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8(word, true) : __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
        return (c & 1 ? v.y : v.x) * scale[i];
    }
    __device__ __forceinline__ v4u column(int c) const {
        v4u f;
#pragma unroll
        for (int d = 0; d < 4; ++d) f[d] = high_halves(__float_as_uint(value(2 * d, c)), __float_as_uint(value(2 * d + 1, c)));
        return f;
    }
};

template <int RT, class Wide>
__device__ __forceinline__ void outer_rows(const LoraOuter &a, const LoraWide &w, const Item &it, float scale, int j0, int col,
                                           bool in, int lane, int wave, v4f (&acc)[RT][8]) {
    const int m = lane & 15, kg = lane >> 4;
    for (int row = it.row0 + wave * kRows; row < it.row1; row += kWaves * kRows) {
        const int r0 = row + kg * 8;
        int token[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) token[i] = token_of(a.row_token, r0 + i, a.T);
        Wide x;
        x.load(w, token, col, in);
        float p[RT][8];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int rank = j0 + j * 16 + m;
#pragma unroll
            for (int i = 0; i < 8; ++i) p[j][i] = w.p[(int64_t)(r0 + i) * a.r + (rank < a.r ? rank : 0)];
        }
        v4u hi[RT], lo[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // a padding row's p must not meet the zeros that stand for its x as a NaN
                const float s0 = token[2 * q] >= 0 ? p[j][2 * q] * scale : 0.0f;
                const float s1 = token[2 * q + 1] >= 0 ? p[j][2 * q + 1] * scale : 0.0f;
                uint32_t h, l;
                split2(s0, s1, h, l);
                hi[j][q] = h, lo[j][q] = l;
            }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const v4u f = x.column(c);
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[j][c] = mfma(lo[j], f, acc[j][c]);
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[j][c] = mfma(hi[j], f, acc[j][c]);
        }
    }
}

// One block: an item's rows, 128 columns of a wide matrix, RT tiles of 16
// ranks.  A lane loads 8 columns of 8 rows and turns them into eight fragments
// with one permutation for every two values, so nothing is staged.  Its waves
// take blocks of 32 rows in turn.
template <int RT, class WideX>
__global__ __launch_bounds__(kBlock) void lora_outer_kernel(const LoraOuter a) {
    __shared__ v4f red[2][RT * 8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, kg = lane >> 4;
    const int per = a.wide[0].slabs + a.wide[1].slabs;
    int at = blockIdx.x % (per * a.passes);
    const Item it = item_of(a, blockIdx.x / (per * a.passes), lane);
    if (it.e < 0 || it.slot >= a.slots) return;          // the whole block
    const int j0 = at / per * RT * 16;
    at %= per;
    const bool second = at >= a.wide[0].slabs;
    const LoraWide &w = a.wide[second ? 1 : 0];
    const int col = (second ? at - a.wide[0].slabs : at) * 128 + m * 8;
    const bool in = col < w.C;
    const float scale = a.scales ? a.scales[it.e] : 1.0f;
    v4f acc[RT][8];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = v4f{0, 0, 0, 0};
    if (second) outer_rows<RT, WideBf16>(a, w, it, scale, j0, col, in, lane, wave, acc);
    else outer_rows<RT, WideX>(a, w, it, scale, j0, col, in, lane, wave, acc);

    // the four waves' sums, always in the same order: (0 + 2) + (1 + 3)
    if (wave >= 2) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) red[wave - 2][i][lane] = acc[i >> 3][i & 7];
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) acc[i >> 3][i & 7] += red[wave][i][lane];
    }
    __syncthreads();
    if (wave == 1) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) red[0][i][lane] = acc[i >> 3][i & 7];
    }
    __syncthreads();
    if (wave != 0 || !in) return;
    const int64_t size = (int64_t)a.r * w.C;
    float *out = it.slot < 0 ? w.out + it.e * size : w.part + it.slot * size;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int rank = j0 + j * 16 + kg * 4;           // four ranks, eight columns
        if (rank >= a.r) continue;
        v4f v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = acc[j][c] + red[0][j * 8 + c][lane];
        if (second) {                                    // [C][r]
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<v4f *>(out + (int64_t)(col + c) * a.r + rank) = v[c];
        } else {                                         // [r][C]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *o = out + (int64_t)(rank + i) * w.C + col;
                *reinterpret_cast<v4f *>(o) = v4f{v[0][i], v[1][i], v[2][i], v[3][i]};
                *reinterpret_cast<v4f *>(o + 4) = v4f{v[4][i], v[5][i], v[6][i], v[7][i]};
            }
        }
    }
}

// The sums of adapters with several items, slots in order; block row y is the
// y-th such adapter
__global__ __launch_bounds__(kBlock) void lora_join_kernel(const LoraOuter a) {
    const int lane = threadIdx.x & 63;
    Scan before{0, 0, 0, 0};
    int e = -1, slot = 0, m = 0;
    for (int e0 = 0; e0 < a.E && e < 0; e0 += 64) {
        int lo, hi;
        const Scan s = scan_adapters(a, e0, lane, before, lo, hi);
        const uint64_t mine = __ballot(s.m > 1 && s.many == (int)blockIdx.y);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            e = e0 + l, slot = __shfl(s.slots, l, 64), m = __shfl(s.m, l, 64);
        }
        before = totals(s);
    }
    if (e < 0 || slot >= a.slots) return;
    const int64_t size0 = (int64_t)a.r * a.wide[0].C, size1 = (int64_t)a.r * a.wide[1].C;
    const int64_t i = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 4;
    if (i >= size0 + size1) return;
    const bool second = i >= size0;
    const LoraWide &w = a.wide[second ? 1 : 0];
    const int64_t size = second ? size1 : size0, at = second ? i - size0 : i;
    const float *p = w.part + slot * size + at;
    v4f v = *reinterpret_cast<const v4f *>(p);
    for (int n = 1; n < m && slot + n < a.slots; ++n) v += *reinterpret_cast<const v4f *>(p + n * size);
    *reinterpret_cast<v4f *>(w.out + e * size + at) = v;
}

template <class Y, int KT>
void start_expand(LoraExpand a, bool wide, hipStream_t stream) {
    const int64_t blocks = a.rows / kRows;
    if (wide) lora_expand_kernel<Y, KT, 4><<<(unsigned)(ceil_div(blocks, 4) * a.tiles), kBlock, 0, stream>>>(a);
    else lora_expand_kernel<Y, KT, 1><<<(unsigned)(blocks * a.tiles), kBlock, 0, stream>>>(a);
}
template <class Y>
void start_expand(const LoraExpand &a, bool wide, hipStream_t stream) {
    if (a.r <= 32) start_expand<Y, 1>(a, wide, stream);
    else if (a.r <= 64) start_expand<Y, 2>(a, wide, stream);
    else start_expand<Y, 4>(a, wide, stream);
}
template <int RT>
void start_outer(const LoraOuter &a, int form, unsigned grid, hipStream_t stream) {
    if (form == 0) lora_outer_kernel<RT, WideBf16><<<grid, kBlock, 0, stream>>>(a);
    else if (form == 1) lora_outer_kernel<RT, WideGrid<false>><<<grid, kBlock, 0, stream>>>(a);
    else lora_outer_kernel<RT, WideGrid<true>><<<grid, kBlock, 0, stream>>>(a);
}

}  // namespace

LoraCut lora_cut(int64_t rows, int64_t K, int cus) {
    // blocks of 32 rows; the wide axis is cut where they alone do not fill the compute units twice, into slices that
    // give every wave of a block a chunk of 128
    const int64_t blocks = rows / kRows, most = ceil_div(K, kWaves * 128);
    int64_t splits = blocks ? ceil_div(2 * cus, blocks) : 1;
    splits = splits < most ? splits : most;
    splits = splits < 16 ? splits : 16;
    const int64_t slice = ceil_div(ceil_div(K, splits), kWaves * 128) * kWaves * 128;
    return {(int)ceil_div(K, slice), (int)slice};
}

hipError_t launch_lora_shrink(const LoraShrink &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.rows / kRows * a.splits);
    if (a.r <= 16) lora_shrink_kernel<1><<<grid, kBlock, 0, stream>>>(a);
    else if (a.r <= 32) lora_shrink_kernel<2><<<grid, kBlock, 0, stream>>>(a);
    else if (a.r <= 64) lora_shrink_kernel<4><<<grid, kBlock, 0, stream>>>(a);
    else lora_shrink_kernel<8><<<grid, kBlock, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_lora_expand(LoraExpand a, bool y_bf16, hipStream_t stream) {
    a.tiles = (int)(a.N ? ceil_div(a.N, 256) : 1);       // N = 0: P alone
    const bool wide = a.rows / kRows * a.tiles >= 16 * (int64_t)device_cu_count();
    if (y_bf16) start_expand<uint16_t>(a, wide, stream);
    else start_expand<float>(a, wide, stream);
    return hipGetLastError();
}

hipError_t launch_lora_transpose(const LoraTranspose &a, hipStream_t stream) {
    int64_t most = 1;
    for (const LoraTranspose::Job &j : a.job) {
        const int64_t n = a.E * ceil_div(j.P, 64) * ceil_div(j.Q, 64);
        most = most > n ? most : n;
    }
    const int64_t cap = 8 * (int64_t)device_cu_count();
    lora_transpose_kernel<<<dim3((unsigned)(most < cap ? most : cap), 2), kBlock, 0, stream>>>(a);
    return hipGetLastError();
}

LoraOuterPlan lora_outer_plan(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N, int cus) {
    const int64_t passes = ceil_div(r, 64), slabs = (ceil_div(K, 128) + ceil_div(N, 128)) * passes;
    const int64_t wanted = slabs < 4 * cus ? 4 * cus / slabs : 1;
    int64_t chunk = ceil_div(ceil_div(rows, wanted), kWaves * kRows) * kWaves * kRows;
    chunk = chunk > 256 ? chunk : 256;
    const int64_t items = rows / chunk + E;
    int64_t slots = 2 * rows / chunk;                    // items of adapters with more than one
    slots = slots < items ? slots : items;
    return {chunk, items, slots};
}

hipError_t launch_lora_outer(LoraOuter a, const LoraOuterPlan &plan, int form, hipStream_t stream) {
    a.chunk = (int)plan.chunk, a.slots = (int)plan.slots;
    for (LoraWide &w : a.wide) w.slabs = (int)ceil_div(w.C, 128);
    a.passes = (int)ceil_div(a.r, 64);
    const unsigned grid = (unsigned)(plan.items * (a.wide[0].slabs + a.wide[1].slabs) * a.passes);
    if (a.r <= 16) start_outer<1>(a, form, grid, stream);
    else if (a.r <= 32) start_outer<2>(a, form, grid, stream);
    else start_outer<4>(a, form, grid, stream);
    if (plan.slots > 1) {
        const int64_t most = plan.slots / 2, many = a.E < most ? a.E : most;
        const int64_t quads = (int64_t)a.r * (a.wide[0].C + a.wide[1].C) / 4;
        lora_join_kernel<<<dim3((unsigned)ceil_div(quads, kBlock), (unsigned)many), kBlock, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mx
