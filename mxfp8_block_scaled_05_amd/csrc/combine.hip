// Expert rows back in token order (the weighted sum of a token's experts) and
// the gradients of that sum.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kBlock = 256;
constexpr int kAhead = 8;          // rows of a token in flight
constexpr int kZeroRows = 8;       // rows a wave looks over for padding

// One 16-byte piece of a row: all of it, or its first n elements and zeros.
template <bool ONCE, class E>
__device__ __forceinline__ v4u load_piece(const E *p, int n) {
    constexpr int kV = Elem<E>::kVec;
    if (n >= kV) return load16<ONCE>(p);
    float f[kV];
    load_head<kV>(p, n, 0.0f, f);
    return Elem<E>::pack(f);                             // exact: the values are the type's own
}
template <class E>
__device__ __forceinline__ void store_piece(E *p, int n, const float *f) {
    constexpr int kV = Elem<E>::kVec;
    if (n >= kV) {
        store16(p, Elem<E>::pack(f));
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = Elem<E>::put(f[i]);
    }
}

// out[t] = sum_j w[t][j] y[pair_row[t][j]], in fp32 and in the order of j,
// rounded once.  HBM-bound: every chosen row is read once.  A thread holds
// one 16-byte piece of one token and asks for it in 8 of the token's rows
// before it adds any: 8192 tokens of 8 x 2048 bf16 take 47.2 us with part of
// y still in the last-level cache; one row after another took 65 us.  ONCE (y
// larger than that cache) reads past it: from HBM 52.5 us (5.8 TB/s) instead of
// 59.4, after a copy that wrote y 151 us for both instead of 160; at 4095
// tokens, where y fits, it would cost 26.8 us instead of 23.8.  Its loads are the row pieces of neighbouring
// threads, so any row length and alignment keeps the rate (1001 columns: 5.2
// TB/s).
template <class E, bool ONCE>
__global__ __launch_bounds__(kBlock) void combine_kernel(const CombineArgs a, int64_t pieces) {
    constexpr int kV = Elem<E>::kVec;
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    const int64_t t = i / pieces;
    if (t >= a.T) return;
    const int64_t col = (i - t * pieces) * kV;
    const int n = (int)(a.H - col < kV ? a.H - col : kV);
    const E *y = static_cast<const E *>(a.y) + col;
    float acc[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        int row[kAhead];
        float w[kAhead];
        v4u r[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            row[u] = j0 + u < a.k ? a.pair_row[t * a.k + j0 + u] : -1;
            w[u] = j0 + u < a.k ? a.w[t * a.k + j0 + u] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (row[u] >= 0 && row[u] < a.rows) r[u] = load_piece<ONCE>(y + row[u] * a.H, n);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (row[u] >= 0 && row[u] < a.rows) {
                float f[kV];
                Elem<E>::unpack(r[u], f);
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[e] = __builtin_fmaf(w[u], f[e], acc[e]);
            }
    }
    store_piece(static_cast<E *>(a.out) + t * a.H + col, n, acc);
}

// W lanes per (token, choice): d_y[row] = w d_out[t] and d_w = <d_out[t],
// y[row]>, the token's d_out row read by its other choices from the cache.
// The blocks after those zero the rows no token owns.  HBM-bound: every row of
// y is read and every row of d_y written once (4095 tokens of 8 x 2048 bf16:
// 52.8 us).  ONCE (both together larger than the last-level cache) keeps them
// out of it: 55.2 us (5.5 TB/s) from HBM instead of 61.7, with the quantizer that
// reads d_y next 182 us instead of 187 (8192 tokens); at 2000 tokens that pair
// would take 52.1 us instead of 46.0.
//
// The lanes and the pieces in flight follow the row's length: 8192 tokens of
// 8 x 200 bf16 take 15.6 us, 25.2 us on whole waves; 8192 x 1 x 64 fp32 3.7
// us, 7.1 us.  Whole strides go without guards (60.4 us with them).  Rows of an odd
// number of bf16 lose a third (8 x 1001: 3.3 TB/s): cutting the pieces at
// multiples of 16 bytes of d_y did not help (109 against 86 us).
template <class E, int W, int U, bool ONCE>
__global__ __launch_bounds__(kBlock) void combine_backward_kernel(const CombineArgs a, int64_t pair_blocks) {
    constexpr int kV = Elem<E>::kVec;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    E *d_y = static_cast<E *>(a.d_y);
    if ((int64_t)blockIdx.x < pair_blocks) {
        const int64_t p = ((int64_t)blockIdx.x * kBlock + threadIdx.x) / W;
        const bool live = p < a.T * a.k;
        const int64_t row = live ? a.pair_row[p] : -1;
        float dot = 0.0f;
        if (row >= 0 && row < a.rows) {
            const float w = a.w[p];
            const E *d = static_cast<const E *>(a.d_out) + p / a.k * a.H;
            const E *y = static_cast<const E *>(a.y) + row * a.H;
            E *dst = d_y + row * a.H;
            int64_t col = (lane & (W - 1)) * kV, base = 0;
            for (; base + U * W * kV <= a.H; base += U * W * kV, col += U * W * kV) {
                v4u rg[U], rf[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rf[u] = load16<ONCE>(y + col + u * W * kV);
                    rg[u] = load16(d + col + u * W * kV);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float g[kV], f[kV];
                    Elem<E>::unpack(rg[u], g);
                    Elem<E>::unpack(rf[u], f);
#pragma unroll
                    for (int e = 0; e < kV; ++e) {
                        dot = __builtin_fmaf(g[e], f[e], dot);
                        g[e] *= w;
                    }
                    store16<ONCE>(dst + col + u * W * kV, Elem<E>::pack(g));
                }
            }
            if (col < a.H) {                             // the rest, in flight together as well
                v4u rg[U], rf[U];
                int n[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = col + u * W * kV;
                    n[u] = (int)(a.H - at < kV ? a.H - at : kV);
                    if (n[u] > 0) {
                        rf[u] = load_piece<ONCE>(y + at, n[u]);
                        rg[u] = load_piece<false>(d + at, n[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (n[u] <= 0) break;
                    float g[kV], f[kV];
                    Elem<E>::unpack(rg[u], g);
                    Elem<E>::unpack(rf[u], f);
#pragma unroll
                    for (int e = 0; e < kV; ++e) {
                        dot = __builtin_fmaf(g[e], f[e], dot);
                        g[e] *= w;
                    }
                    store_piece(dst + col + u * W * kV, n[u], g);
                }
            }
        }
        dot = group_reduce<W>(dot, OpAdd());
        if (live && (lane & (W - 1)) == 0) a.d_w[p] = dot;
        return;
    }
    const int64_t base = (((int64_t)blockIdx.x - pair_blocks) * (kBlock / 64) + wave) * kZeroRows;
    const int64_t mine = base + lane;
    bool empty = false;
    if (lane < kZeroRows && mine < a.rows) {
        const int64_t t = a.row_token[mine];
        empty = t < 0 || t >= a.T;
    }
    float zero[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) zero[e] = 0.0f;
    for (uint64_t m = __ballot(empty); m; m &= m - 1) {
        const int64_t row = base + __builtin_ctzll(m);
        for (int64_t col = lane * kV; col < a.H; col += 64 * kV)
            store_piece(d_y + row * a.H + col, (int)(a.H - col < kV ? a.H - col : kV), zero);
    }
}

}  // namespace

hipError_t launch_combine(const CombineArgs &a, bool bf16, hipStream_t stream) {
    const int64_t pieces = ceil_div(a.H, bf16 ? 8 : 4);
    const unsigned grid = (unsigned)ceil_div(a.T * pieces, kBlock);
    const bool once = a.rows * a.H * (bf16 ? 2 : 4) > kLastLevelBytes;
    if (bf16) {
        if (once) combine_kernel<uint16_t, true><<<grid, kBlock, 0, stream>>>(a, pieces);
        else combine_kernel<uint16_t, false><<<grid, kBlock, 0, stream>>>(a, pieces);
    } else {
        if (once) combine_kernel<float, true><<<grid, kBlock, 0, stream>>>(a, pieces);
        else combine_kernel<float, false><<<grid, kBlock, 0, stream>>>(a, pieces);
    }
    return hipGetLastError();
}

template <class E, int W, int U>
static void start_backward(const CombineArgs &a, hipStream_t stream) {
    const int64_t pair_blocks = ceil_div(a.T * a.k, kBlock / W);
    const unsigned grid = (unsigned)(pair_blocks + ceil_div(a.rows, kBlock / 64 * kZeroRows));
    if (2 * a.rows * a.H * (int64_t)sizeof(E) > kLastLevelBytes)
        combine_backward_kernel<E, W, U, true><<<grid, kBlock, 0, stream>>>(a, pair_blocks);
    else
        combine_backward_kernel<E, W, U, false><<<grid, kBlock, 0, stream>>>(a, pair_blocks);
}
template <class E>
static void start_backward(const CombineArgs &a, hipStream_t stream) {
    const int64_t pieces = ceil_div(a.H, Elem<E>::kVec);             // of a row
    if (pieces <= 16) start_backward<E, 16, 1>(a, stream);
    else if (pieces <= 32) start_backward<E, 32, 1>(a, stream);
    else if (pieces <= 64) start_backward<E, 64, 1>(a, stream);
    else if (pieces <= 128) start_backward<E, 64, 2>(a, stream);
    else start_backward<E, 64, 4>(a, stream);
}

hipError_t launch_combine_backward(const CombineArgs &a, bool bf16, hipStream_t stream) {
    if (bf16) start_backward<uint16_t>(a, stream);
    else start_backward<float>(a, stream);
    return hipGetLastError();
}

}  // namespace mx
