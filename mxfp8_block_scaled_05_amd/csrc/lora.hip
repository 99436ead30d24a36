// Low-rank adapters of many requests beside a shared projection: y += s B (A x)
// for rows sorted by adapter, and the gradients of x, A and B.
//
// A group's rows start at a multiple of 32, so every block of 32 sorted rows
// has one adapter and its products run on the matrix unit.  The rank is small:
// every product reads or writes one wide matrix once, and what bounds it is how
// that matrix moves.  Operands are loaded in runs of a row and turned in LDS or
// in registers; the weights and P come from the caches.
//
//   shrink   P = X A^T          partial sums over slices of the wide axis
//   expand   Y += (s P) B^T     sums the partials, keeps P
//   outer    W = (s P)^T X      sums over rows, per adapter
// Forward: shrink (x, A), expand (y, B).  Backward, with the transposed weights:
// shrink (d_y, B^T), expand (d_x, A^T), outer twice (d_a: S and x; d_b: hidden
// and d_y).
//
// P is held in fp32.  Where it is an operand of the matrix unit it enters as a
// sum of bf16 numbers: three, which hold all 24 bits, where the result is fp32
// (y, the weights' gradients), two, which lose 2^-16 of the value, where it is
// rounded to bf16 (2^-8).  The products of the parts cost matrix time that is
// idle anyway: these kernels wait for memory.
//
// The parts of a finite P may be 0 or differ in sign, so against an infinity, or
// where a product leaves fp32, they make a NaN of what is an infinity.  The
// first part alone, which has P's sign and is 0 only with it, decides there: a
// NaN among the sums has its tile's products taken again with that part (the
// gradients of 8192 rows with an infinity in x, d_y or b 178 to 194 us for 99).
#include <type_traits>

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

// Two values as a sum of N pairs of bf16, each pair in a word, the largest
// first.  A finite value that bf16 would round to infinity begins with bf16's
// largest number instead; an infinity or NaN has no rest.
constexpr float kLargestBf16 = 0x1.FEp127f;
__device__ __forceinline__ float in_range(float v) {
    return __builtin_isfinite(v) ? __builtin_amdgcn_fmed3f(v, -kLargestBf16, kLargestBf16) : v;
}
__device__ __forceinline__ float rest_of(float v, float taken) {
    const float d = v - taken;
    return d == d ? d : 0.0f;
}
template <int N>
__device__ __forceinline__ void split_pair(float v0, float v1, uint32_t (&out)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        out[n] = n == 0 ? bf16x2_rne(in_range(v0), in_range(v1)) : bf16x2_rne(v0, v1);
        v0 = rest_of(v0, __uint_as_float(out[n] << 16));
        v1 = rest_of(v1, __uint_as_float(out[n] & 0xFFFF0000u));
    }
}

// Whether one of a lane's sums is a NaN; four sums with those of `first` in
// such places
template <int N>
__device__ __forceinline__ bool has_nan(const v4f (&d)[N]) {
    bool nan = false;
#pragma unroll
    for (int n = 0; n < N; ++n) nan = nan || __builtin_isunordered(d[n].x, d[n].y) || __builtin_isunordered(d[n].z, d[n].w);
    return nan;
}
__device__ __forceinline__ v4f instead_of_nan(v4f d, v4f first) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = d[i] == d[i] ? d[i] : first[i];
    return d;
}

// The compiler moves a load to where its value is first used, a round later,
// unless it must not.
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }

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

// The token that a row's entry names, -1 for padding
__device__ __forceinline__ int token_of(int64_t t, int64_t T) { return t >= 0 && t < T ? (int)t : -1; }

// ---------------------------------------------------------------- shrink

// One block: 32 sorted rows, a slice of the wide axis, all ranks.  Its waves
// take chunks of it in turn, each on its own.  RT: tiles of 16 ranks.  Bound by
// loads in flight: 8192 rows of 4096, rank 64, by itself 28 us (67 MB, 2.4 TB/s;
// 11 us of it the launch, the first loads and the join).
//
// The matrix unit wants 16 rows from 16 neighbouring lanes, and a load that is
// laid out so touches 16 cache lines with every 256 bytes it brings (8192 rows
// of 6144: 34 us, 10 bytes a clock from a compute unit's cache).  So both
// operands are loaded in runs of 256 or 128 bytes of a row, kept in registers
// until the chunk before is used, and turned in the wave's part of LDS: row r's
// 16-byte piece c lies at c ^ r, which spreads 16 rows over the banks.
template <int RT, int WAVES>
struct ShrinkShape {
    static constexpr int kChunk = RT == 1 || (RT == 2 && WAVES == 4) ? 128 : 64;         // columns of a wave's chunk
    static constexpr int kPieces = kChunk / 8;                   // 16-byte pieces of a row of it
    static constexpr int kPass = 64 / kPieces;                   // rows that a wave loads at once
    static constexpr int kX = kRows / kPass, kW = RT * 16 / kPass;
    static constexpr int kWaveBytes = (kRows + RT * 16) * kChunk * 2;
    static constexpr int kRedBytes = WAVES * kRows * RT * 64;
    static constexpr int kBytes = WAVES * kWaveBytes > kRedBytes ? WAVES * kWaveBytes : kRedBytes;
};

// Columns [k_first, k1) of block rb's rows against its adapter's weights: the
// waves' sums in `room`, [WAVES][32][RT * 4], four ranks each.  Whether the rows
// have an adapter is the same for the whole block.
template <int RT, int WAVES>
__device__ __forceinline__ bool shrink_rows(const LoraShrink &a, int rb, int k_first, int k1, v4u *room) {
    using S = ShrinkShape<RT, WAVES>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, kg = lane >> 4;
    const int piece = lane % S::kPieces, sub = lane / S::kPieces;
    int64_t named[S::kX];                                // asked for beside the offsets, not after them
#pragma unroll
    for (int i = 0; i < S::kX; ++i) named[i] = a.row_token[(int64_t)rb * kRows + i * S::kPass + sub];
    const int e = adapter_of(a.offsets, a.E, rb * kRows, lane);
    if (e < 0 || e >= a.E) return false;
    // Rows of padding are loaded from row 0 and ranks past r from rank 0: what they give is not kept, and loads that
    // nothing branches around let the compiler wait for the oldest alone.
    const uint16_t *x[S::kX], *w[S::kW];
#pragma unroll
    for (int i = 0; i < S::kX; ++i) {
        const int token = token_of(named[i], a.T);
        x[i] = a.x + (token < 0 ? 0 : token) * a.ld + piece * 8;
    }
#pragma unroll
    for (int i = 0; i < S::kW; ++i) {
        const int rank = i * S::kPass + sub;
        w[i] = a.w + ((int64_t)e * a.r + (rank < a.r ? rank : 0)) * a.K + piece * 8;
    }
    v4f acc[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[t][j] = v4f{0, 0, 0, 0};

    v4u xs[S::kX], ws[S::kW];
    auto ask = [&](int k0) {
#pragma unroll
        for (int i = 0; i < S::kX; ++i) xs[i] = *reinterpret_cast<const v4u *>(x[i] + k0);
#pragma unroll
        for (int i = 0; i < S::kW; ++i) ws[i] = *reinterpret_cast<const v4u *>(w[i] + k0);
    };
    auto ask_end = [&](int k0) {                         // the columns below k1 and zeros
        const bool in = k0 + piece * 8 < k1;
        const int64_t back = in ? k0 : -piece * 8;
#pragma unroll
        for (int i = 0; i < S::kX; ++i) {
            const v4u v = *reinterpret_cast<const v4u *>(x[i] + back);
            xs[i] = in ? v : v4u{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < S::kW; ++i) {
            const v4u v = *reinterpret_cast<const v4u *>(w[i] + back);
            ws[i] = in ? v : v4u{0, 0, 0, 0};
        }
    };
    v4u *mine = room + wave * (S::kWaveBytes / 16);
    auto slot = [&](int row, int c) { return row * S::kPieces + (c ^ (row % S::kPieces)); };
    auto turn = [&]() {
#pragma unroll
        for (int i = 0; i < S::kX; ++i) mine[slot(i * S::kPass + sub, piece)] = xs[i];
#pragma unroll
        for (int i = 0; i < S::kW; ++i) mine[slot(kRows + i * S::kPass + sub, piece)] = ws[i];
        wave_sync();
    };
    auto use = [&]() {
#pragma unroll
        for (int s = 0; s < S::kChunk / 32; ++s) {
            v4u wf[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j) wf[j] = mine[slot(kRows + j * 16 + m, s * 4 + kg)];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const v4u xf = mine[slot(t * 16 + m, s * 4 + kg)];
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[t][j] = mfma(wf[j], xf, acc[t][j]);
            }
        }
        wave_sync();
    };
    constexpr int kStep = WAVES * S::kChunk;
    int k0 = k_first + wave * S::kChunk;
    if (k0 + S::kChunk <= k1) {
        ask(k0);
        for (; k0 + S::kChunk <= k1; k0 += kStep) {
            turn();
            ask(k0 + kStep + S::kChunk <= k1 ? k0 + kStep : k0);         // the last time for nothing
            keep_order();
            use();
        }
    }
    if (k0 < k1) {
        ask_end(k0);
        turn();
        use();
    }
    // a lane holds four ranks, 4 kg.., of row m
    __syncthreads();
    auto red = reinterpret_cast<v4f (*)[kRows][RT * 4]>(room);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < RT; ++j) red[wave][t * 16 + m][j * 4 + kg] = acc[t][j];
    __syncthreads();
    return true;
}

template <int RT>
__global__ __launch_bounds__(kBlock) void lora_shrink_kernel(const LoraShrink a) {
    __shared__ v4u room[ShrinkShape<RT, kWaves>::kBytes / 16];
    const int rb = blockIdx.x / a.splits, split = blockIdx.x - rb * a.splits;
    if (!shrink_rows<RT, kWaves>(a, rb, split * a.slice, min(a.K, (split + 1) * a.slice), room)) return;
    auto red = reinterpret_cast<v4f (*)[kRows][RT * 4]>(room);
    float *out = a.part + ((int64_t)split * a.rows + (int64_t)rb * kRows) * a.r;
    for (int i = threadIdx.x; i < kRows * RT * 4; i += kBlock) {
        const int row = i / (RT * 4), q = i - row * (RT * 4);
        if (q * 4 >= a.r) continue;
        v4f v = red[0][row][q];
#pragma unroll
        for (int n = 1; n < kWaves; ++n) v += red[n][row][q];
        if (token_of(a.row_token[(int64_t)rb * kRows + row], a.T) < 0) v = v4f{0, 0, 0, 0};
        *reinterpret_cast<v4f *>(out + (int64_t)row * a.r + q * 4) = v;
    }
}

// P as the outer products take it: for every 32 rows and 16 ranks three
// fragments, a lane's 8 rows of one rank, 1 KB each.
constexpr int kOuterParts = 3;
__device__ __forceinline__ void pack_rows(const float (&p)[8], v4u *out) {
    v4u parts[kOuterParts];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t word[kOuterParts];
        split_pair(p[2 * q], p[2 * q + 1], word);
#pragma unroll
        for (int n = 0; n < kOuterParts; ++n) parts[n][q] = word[n];
    }
#pragma unroll
    for (int n = 0; n < kOuterParts; ++n) out[n * 64] = parts[n];
}

// ---------------------------------------------------------------- expand

// y in 16-byte pieces: of a row's 64 columns, those that a wave loads of so
// many rows at once
template <class Y>
struct Tile {
    static constexpr int kVec = 16 / sizeof(Y), kPieces = 64 / kVec, kPass = 64 / kPieces, kPasses = 16 / kPass;
    __device__ static __forceinline__ v4u add(v4u y, const float *d) {
        float f[kVec];
        Elem<Y>::unpack(y, f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] += d[i];
        return Elem<Y>::pack(f);
    }
};

// One block: RB groups of 32 sorted rows; its waves go through their columns
// 64 at a time, `step` apart.  The products of 16 rows are taken as B P^T and
// turned in the wave's part of LDS, so that y is read and written in runs of
// 128 or 256 bytes (in the matrix unit's own layout 16 neighbouring lanes hold
// 16 rows, 16 cache lines for 256 bytes).  The next columns' y and B are asked
// for before the current ones are used.  Joining P once for many columns
// matters: 8192 rows of rank 64 to 6144 take 60 us with P joined for every 256.
// Whole calls with inputs that change: 8192 rows of rank 128, 4096 to 6144, 105 us
// with bf16 y and 139 with fp32; 16384 rows of rank 64 140 and 213.
// KT: steps of 32 ranks.  LOOP: several columns.  By itself rank 64 to 8192 x 6144
// takes 51 us, rank 32 to 8192 x 4096 31 us; y alone, read and written in place
// (201 MB), takes 37.4 at its best.
//
// B's rows are r long, so 64 of them are one run of memory.  Above rank 32 they
// are loaded as such and turned in LDS; loaded straight into fragments they
// would touch a cache line for every 16 bytes (twice the time of y itself).
template <class Y, int KT, int RB, int WAVES>
struct ExpandShape {
    static constexpr int kParts = sizeof(Y) == 4 ? 3 : 2;
    static constexpr bool kTurnB = KT > 1;
    static constexpr int kB = 4 * KT;                            // 16-byte pieces of a row of B, and of a lane's B
    typedef v4u Frag[RB * 2][KT][kParts][64];                    // P of each 16 rows as the matrix unit takes it, in parts
    typedef float Turn[WAVES][16][68];                           // 4 more than a row: 16 rows on all banks
    static constexpr int kBs = kTurnB ? WAVES * 64 * kB : 1;     // pieces of B
};
// sum(row, j, v): P of a row of the block, ranks j to j + 7
template <class Y, int KT, int RB, bool LOOP, int WAVES, class Sum>
__device__ __forceinline__ void expand_rows(const LoraExpand &a, int group, int tile0,
                                            typename ExpandShape<Y, KT, RB, WAVES>::Frag &frag,
                                            typename ExpandShape<Y, KT, RB, WAVES>::Turn &turn, v4u *bs, Sum sum) {
    using T = Tile<Y>;
    using S = ExpandShape<Y, KT, RB, WAVES>;
    constexpr int kParts = S::kParts, kPasses = T::kPasses, kB = S::kB;
    constexpr bool kTurnB = S::kTurnB;
    // scaled P of the block's rows, first 64 ranks and the rest, before what `turn` and `bs` are for
    auto flat = reinterpret_cast<float (*)[68]>(&turn[0][0][0]);
    auto upper = reinterpret_cast<float (*)[68]>(&bs[0]);
    static_assert(RB * 32 * 68 * 4 <= sizeof(turn) && (KT < 4 || RB * 32 * 68 * 4 <= S::kBs * 16), "P's rows fit");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, kg = lane >> 4;
    const int rb0 = group * RB;
    const int blocks = (int)(a.rows / kRows);
    const int piece = lane % T::kPieces, sub = lane / T::kPieces;
    // asked for beside the offsets, not after them
    int64_t named[RB * 2][kPasses];
#pragma unroll
    for (int i = 0; i < RB * 2; ++i)
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int64_t row = (int64_t)rb0 * kRows + i * 16 + p * T::kPass + sub;
            named[i][p] = a.row_token[row < a.rows ? row : 0];
        }
    int e[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        e[i] = adapter_of(a.offsets, a.E, (rb0 + i) * kRows, lane);
        if (e[i] >= a.E || rb0 + i >= blocks) e[i] = -1;
    }
    int token[RB * 2][kPasses];
#pragma unroll
    for (int i = 0; i < RB * 2; ++i)
#pragma unroll
        for (int p = 0; p < kPasses; ++p) token[i][p] = e[i >> 1] < 0 ? -1 : token_of(named[i][p], a.T);

    struct Ahead {
        v4u y[RB * 2][kPasses];
        v4u b[kTurnB ? 1 : kB];                          // fragments [q]
    };
    v4u run[kTurnB ? kB : 1];                            // or the run's pieces: one set, in LDS before the next is asked for
    v4u *mine = bs + wave * 64 * kB;
    auto slot = [&](int n, int c) { return n * kB + (c ^ (n % (kB < 16 ? kB : 16))); };
    int b_slot[kTurnB ? kB : 1], b_piece[kTurnB ? kB : 1];
    if constexpr (kTurnB) {
        const int per = a.r / 8;                         // pieces of a row
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int at = i < per ? i * 64 + lane : lane;               // pieces that there are not: the first again
            b_piece[i] = at;
            b_slot[i] = slot(at / per, at % per);
        }
    }
    auto clear_b = [&]() {                               // ranks past r
        if constexpr (kTurnB) {
#pragma unroll
            for (int i = 0; i < kB; ++i) mine[i * 64 + lane] = v4u{0, 0, 0, 0};
            wave_sync();
        }
    };
    // All 64 rows have a token, one adapter and whole columns: nothing is branched around, so that the compiler counts
    // what is in flight and waits for the oldest alone.  Otherwise rows of padding and columns past N are loaded from
    // row 0 and column 0 and not stored.
    bool whole = a.N % 64 == 0;
#pragma unroll
    for (int i = 0; i < RB * 2; ++i)
#pragma unroll
        for (int p = 0; p < kPasses; ++p) whole = whole && __ballot(token[i][p] >= 0) == ~0ull && e[i >> 1] == e[0];
    auto place = [&](int i, int p, int c0) {
        const int col = c0 + piece * T::kVec;
        return static_cast<Y *>(a.y) + (token[i][p] < 0 ? 0 : token[i][p]) * a.ld + (col < a.N ? col : 0);
    };
    auto ask = [&](Ahead &n, int adapter, int c0) {
        const uint16_t *w = a.w + ((int64_t)adapter * a.N + c0) * a.r;
        if constexpr (kTurnB) {
            const int pieces = min(a.N - c0, 64) * (a.r / 8);
#pragma unroll
            for (int i = 0; i < kB; ++i) run[i] = *reinterpret_cast<const v4u *>(w + (b_piece[i] < pieces ? b_piece[i] : 0) * 8);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = q * 16 + m, j = kg * 8;
                const v4u v = *reinterpret_cast<const v4u *>(w + (c0 + col < a.N ? col : 0) * a.r + (j < a.r ? j : 0));
                n.b[q] = j < a.r ? v : v4u{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < RB * 2; ++i)
#pragma unroll
            for (int p = 0; p < kPasses; ++p) n.y[i][p] = *reinterpret_cast<const v4u *>(place(i, p, c0));
    };
    auto turn_b = [&]() {
        if constexpr (kTurnB) {
#pragma unroll
            for (int i = 0; i < kB; ++i) mine[b_slot[i]] = run[i];
            wave_sync();
        }
    };
    auto use = [&](auto whole_rows, const Ahead &n, int adapter, int c0) {
        constexpr bool kWhole = decltype(whole_rows)::value;
        const bool in = c0 + piece * T::kVec < a.N;
#pragma unroll
        for (int i = 0; i < RB * 2; ++i) {
            if constexpr (!kWhole) {
                bool any = false;
#pragma unroll
                for (int p = 0; p < kPasses; ++p) any = any || __ballot(token[i][p] >= 0) != 0;
                if (!any || e[i >> 1] != adapter) continue;
            }
            v4f d[4] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                v4u b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = kTurnB ? mine[slot(q * 16 + m, kt * 4 + kg)] : n.b[q];
#pragma unroll
                for (int s = kParts - 1; s >= 0; --s) {
                    const v4u p = frag[i][kt][s][lane];
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[q] = mfma(b[q], p, d[q]);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<v4f *>(&turn[wave][m][q * 16 + kg * 4]) = d[q];
            if (__builtin_expect(__ballot(has_nan(d)) != 0, 0)) {
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    v4f first = {0, 0, 0, 0};
#pragma unroll 1
                    for (int kt = 0; kt < KT; ++kt) {
                        v4u b;
                        if constexpr (kTurnB) b = mine[slot(q * 16 + m, kt * 4 + kg)];
                        else b = q == 0 ? n.b[0] : q == 1 ? n.b[1] : q == 2 ? n.b[2] : n.b[3];
                        first = mfma(b, frag[i][kt][0][lane], first);
                    }
                    auto sums = reinterpret_cast<v4f *>(&turn[wave][m][q * 16 + kg * 4]);          // this lane's
                    *sums = instead_of_nan(*sums, first);
                }
            }
            wave_sync();
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                float f[T::kVec];
#pragma unroll
                for (int v = 0; v < T::kVec; v += 4) {
                    const v4f u = *reinterpret_cast<const v4f *>(&turn[wave][p * T::kPass + sub][piece * T::kVec + v]);
                    f[v] = u.x, f[v + 1] = u.y, f[v + 2] = u.z, f[v + 3] = u.w;
                }
                if (kWhole || (in && token[i][p] >= 0)) *reinterpret_cast<v4u *>(place(i, p, c0)) = T::add(n.y[i][p], f);
            }
            wave_sync();
        }
    };
    auto columns = [&](auto whole_rows, Ahead (&n)[1 + LOOP], int adapter, int c0, int step) {
        if constexpr (!LOOP) {
            if (c0 >= a.N) return;
            turn_b();
            use(whole_rows, n[0], adapter, c0);
        } else {
            for (; c0 < a.N; c0 += 2 * step) {
                turn_b();
                ask(n[1], adapter, c0 + step < a.N ? c0 + step : c0);    // the last time for nothing
                keep_order();
                use(whole_rows, n[0], adapter, c0);
                if (c0 + step >= a.N) break;
                turn_b();
                ask(n[0], adapter, c0 + 2 * step < a.N ? c0 + 2 * step : c0 + step);
                keep_order();
                use(whole_rows, n[1], adapter, c0 + step);
            }
        }
    };
    const int first = (tile0 * WAVES + wave) * 64, step = a.step * WAVES * 64;
    int start = 0;                                       // the first group that has an adapter
#pragma unroll
    for (int i = RB - 1; i >= 0; --i) start = e[i] >= 0 ? i : start;
    const int lead = e[start];
    Ahead ahead[1 + LOOP];
    if (lead >= 0 && first < a.N) ask(ahead[0], lead, first);

    for (int i = threadIdx.x; i < RB * 2 * KT * 64; i += WAVES * 64) {
        const int l = i & 63, kt = (i >> 6) % KT, mt = (i >> 6) / KT;
        const int ee = RB == 1 || mt < 2 ? e[0] : e[RB - 1];
        const int64_t row = (int64_t)rb0 * kRows + mt * 16 + (l & 15);
        const int j = kt * 32 + (l >> 4) * 8;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const bool in = j < a.r && row < a.rows;
        if (in && ee >= 0) sum(row, j, v);
        if (a.hidden && tile0 == 0 && in) {
            float *h = a.hidden + row * a.r + j;
            *reinterpret_cast<v4f *>(h) = v4f{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<v4f *>(h + 4) = v4f{v[4], v[5], v[6], v[7]};
        }
        const float scale = a.scales && ee >= 0 ? a.scales[ee] : 1.0f;
        v4u parts[kParts];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t word[kParts];
            split_pair(v[2 * q] * scale, v[2 * q + 1] * scale, word);
#pragma unroll
            for (int n = 0; n < kParts; ++n) parts[n][q] = word[n];
        }
#pragma unroll
        for (int n = 0; n < kParts; ++n) frag[mt][kt][n][l] = parts[n];
        if (a.packed && tile0 == 0) {                    // for the outer products below, by way of LDS; half of rank 128 at a time
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = ee >= 0 ? v[q] * scale : 0.0f;
            if (j < 64) {
                *reinterpret_cast<v4f *>(&flat[mt * 16 + (l & 15)][j]) = v4f{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<v4f *>(&flat[mt * 16 + (l & 15)][j + 4]) = v4f{v[4], v[5], v[6], v[7]};
            } else {
                *reinterpret_cast<v4f *>(&upper[mt * 16 + (l & 15)][j - 64]) = v4f{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<v4f *>(&upper[mt * 16 + (l & 15)][j - 60]) = v4f{v[4], v[5], v[6], v[7]};
            }
        }
    }
    __syncthreads();
    if (a.packed && tile0 == 0) {
        const int tiles = (a.r + 15) / 16;
        for (int i = wave; i < RB * tiles; i += WAVES) {
            const int rb = rb0 + i / tiles, jt = i % tiles;
            if (rb >= blocks) break;
            float p[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int row = (rb - rb0) * kRows + kg * 8 + q;
                p[q] = jt < 4 ? flat[row][jt * 16 + m] : upper[row][jt * 16 - 64 + m];
            }
            pack_rows(p, a.packed + ((int64_t)rb * tiles + jt) * kOuterParts * 64 + lane);
        }
        __syncthreads();
    }
    clear_b();
    // groups of one adapter together, one after another where they differ
#pragma unroll
    for (int s = 0; s < RB; ++s) {
        const int adapter = e[s];
        if (adapter < 0 || (s && adapter == e[s - 1])) continue;
        if (s != start && first < a.N) ask(ahead[0], adapter, first);
        if (whole) columns(std::true_type(), ahead, adapter, first, step);
        else columns(std::false_type(), ahead, adapter, first, step);
    }
}

template <class Y, int KT, int RB, bool LOOP>
__global__ __launch_bounds__(kBlock, KT == 4 ? 1 : 2) void lora_expand_kernel(const LoraExpand a) {
    using S = ExpandShape<Y, KT, RB, kWaves>;
    __shared__ typename S::Frag frag;
    __shared__ typename S::Turn turn;
    __shared__ v4u bs[S::kBs];
    const int group = blockIdx.x / a.step;
    expand_rows<Y, KT, RB, LOOP, kWaves>(a, group, blockIdx.x - group * a.step, frag, turn, bs, [&](int64_t row, int j, float (&v)[8]) {
        const float *p = a.part + row * a.r + j;
        for (int s = 0; s < a.splits; ++s, p += a.rows * a.r) {
            const v4f lo = *reinterpret_cast<const v4f *>(p), hi = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += lo[q], v[4 + q] += hi[q];
        }
    });
}

// Both in one launch: each block takes the whole product with A of its 32 rows,
// and its share of the columns of y.  Blocks beside each other on the same rows
// take that product each for itself.  The sums over ranks stay in LDS (no
// partials in memory), and eight waves join them once.  8192 rows of rank 64, 4096
// to 6144: 56 us on one input, 73 with inputs that change (270 MB, 3.7 TB/s), and
// 105 where y is fp32 (470 MB, 4.5 TB/s): a compute unit's waves first all read x
// and then all update y.
constexpr int kBothWaves = 8;
template <class Y, int RT>
__global__ __launch_bounds__(kBothWaves * 64) void lora_both_kernel(const LoraShrink s, const LoraExpand a) {
    constexpr int KT = RT == 4 ? 2 : 1;
    using S = ExpandShape<Y, KT, 1, kBothWaves>;
    constexpr int kRoom = ShrinkShape<RT, kBothWaves>::kBytes / 16;
    __shared__ v4u room[kRoom > S::kBs ? kRoom : S::kBs];        // the sums, then B
    __shared__ typename S::Frag frag;
    __shared__ typename S::Turn turn;
    const int rb = blockIdx.x / a.step;
    shrink_rows<RT, kBothWaves>(s, rb, 0, s.K, room);
    auto red = reinterpret_cast<const v4f (*)[kRows][RT * 4]>(room);
    expand_rows<Y, KT, 1, true, kBothWaves>(a, rb, blockIdx.x - rb * a.step, frag, turn, room, [&](int64_t row, int j, float (&v)[8]) {
        if (j >= RT * 16 || token_of(a.row_token[row], a.T) < 0) return;
        const int at = (int)(row - (int64_t)rb * kRows);
        for (int n = 0; n < kBothWaves; ++n) {
            const v4f lo = red[n][at][j >> 2], hi = red[n][at][(j >> 2) + 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += lo[q], v[4 + q] += hi[q];
        }
    });
}

// ---------------------------------------------------------------- before the gradients

// The weights transposed, [E][P][Q] -> [E][Q][P] in 64 x 64 tiles (P and Q
// multiples of 8), and the hidden rows, scaled, as the outer products take them.
// A small launch: 4 to 5 us.
__global__ __launch_bounds__(kBlock) void lora_prepare_kernel(const LoraPrepare a) {
    __shared__ uint16_t t[64][72];
    if (blockIdx.y == 2) {
        const int lane = threadIdx.x & 63, m = lane & 15, kg = lane >> 4;
        const int tiles = (a.r + 15) / 16;
        const int64_t all = a.rows / kRows * tiles;
        for (int64_t i = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * kWaves) {
            const int64_t rb = i / tiles;
            const int rank = (int)(i - rb * tiles) * 16 + m;
            float p[8];
            int64_t named[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int64_t row = rb * kRows + kg * 8 + q;
                p[q] = a.hidden[row * a.r + (rank < a.r ? rank : 0)];
                named[q] = a.row_token[row];
            }
            const int e = adapter_of(a.offsets, a.E, (int)rb * kRows, lane);
            const bool in = e >= 0 && e < a.E && rank < a.r;
            const float scale = in && a.scales ? a.scales[e] : 1.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) p[q] = in && token_of(named[q], a.T) >= 0 ? p[q] * scale : 0.0f;
            pack_rows(p, a.packed + i * kOuterParts * 64 + lane);
        }
        return;
    }
    const LoraPrepare::Job &job = a.job[blockIdx.y];
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
// load() only asks: what is done with the values waits for settle().
struct WideBf16 {
    v4u r[8];
    uint32_t real;                                       // bit i: row i has a token
    __device__ __forceinline__ void load(const LoraWide &w, const int *token, int col, bool in) {
        real = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool has = token[i] >= 0 && in;
            real |= has ? 1u << i : 0u;
            r[i] = *reinterpret_cast<const v4u *>(static_cast<const uint16_t *>(w.x) + (has ? token[i] * w.ld + col : 0));
        }
    }
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = real >> i & 1 ? r[i] : v4u{0, 0, 0, 0};
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
    uint8_t code[8];
    float scale[8];
    uint32_t real;
    __device__ __forceinline__ void load(const LoraWide &w, const int *token, int col, bool in) {
        const uint8_t *x = static_cast<const uint8_t *>(w.x);
        real = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool has = token[i] >= 0 && in;
            const int t = has ? token[i] : 0, c = has ? col : 0;
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
            real |= has ? 1u << i : 0u;
            q[i] = *reinterpret_cast<const v2i *>(x + at);
            code[i] = w.s[sat];
        }
    }
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = code[i];
            const bool has = real >> i & 1;
            q[i] = has ? q[i] : v2i{0, 0};
            scale[i] = bits_to_float(!has ? 0u : c == 0u ? 0x00400000u : c == 255u ? 0x7FC00000u : c << 23);
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
__device__ __forceinline__ void outer_rows(const LoraOuter &a, const LoraWide &w, const Item &it, int jt0, int col, bool in, int lane,
                                           int wave, v4f (&acc)[RT][8]) {
    const int kg = lane >> 4, tiles = (a.r + 15) / 16;
    constexpr int kStep = kWaves * kRows;
    // While a block of 32 rows is used, the next one's values and the tokens of the one after it are on their way.
    int64_t named[8];
    auto ask_tokens = [&](int row) {
#pragma unroll
        for (int i = 0; i < 8; ++i) named[i] = a.row_token[row < it.row1 ? row + kg * 8 + i : 0];
    };
    auto take_tokens = [&](int row, int (&token)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) token[i] = named[i] >= 0 && named[i] < a.T && row < it.row1 ? (int)named[i] : -1;
    };
    auto ask_p = [&](int row, v4u (&p)[RT][kOuterParts]) {
        row = row < it.row1 ? row : it.row0;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int jt = jt0 + j < tiles ? jt0 + j : jt0;              // ranks that there are not: not kept
            const v4u *from = w.p + ((int64_t)(row >> 5) * tiles + jt) * kOuterParts * 64 + lane;
#pragma unroll
            for (int n = 0; n < kOuterParts; ++n) p[j][n] = from[n * 64];
        }
    };
    auto use = [&](Wide &x, const v4u (&p)[RT][kOuterParts]) {
        x.settle();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const v4u f = x.column(c);
#pragma unroll
            for (int n = kOuterParts - 1; n >= 0; --n)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[j][c] = mfma(p[j][n], f, acc[j][c]);
        }
    };
    Wide x[2];
    int token[2][8];
    int row = it.row0 + wave * kRows;
    // An item without rows may belong to a call without any: nothing at all is read then.  Behind an item's last rows
    // row 0 of the tables and of x stands in for what would be next.
    if (row >= it.row1) return;
    // Loads come back in the order of their asking, so the tokens are asked for first: the values that need them must
    // not have to wait for the values before.
    v4u p[2][RT][kOuterParts];
    ask_tokens(row);
    take_tokens(row, token[0]);
    ask_tokens(row + kStep);
    ask_p(row, p[0]);
    x[0].load(w, token[0], col, in);
    for (; row < it.row1; row += 2 * kStep) {
        take_tokens(row + kStep, token[1]);
        ask_tokens(row + 2 * kStep);
        ask_p(row + kStep, p[1]);
        x[1].load(w, token[1], col, in);
        keep_order();
        use(x[0], p[0]);
        if (row + kStep >= it.row1) break;
        take_tokens(row + 2 * kStep, token[0]);
        ask_tokens(row + 3 * kStep);
        ask_p(row + 2 * kStep, p[0]);
        x[0].load(w, token[0], col, in);
        keep_order();
        use(x[1], p[1]);
    }
}

// Where the item's sums at `out` are NaN: those of P's first parts alone.  By
// the wave that wrote them, over all of the item's rows.
template <int RT, class Wide, bool SECOND>
__device__ __forceinline__ void outer_first(const LoraOuter &a, const LoraWide &w, const Item &it, int j0, int col, bool in, int lane,
                                            float *out) {
    const int kg = lane >> 4, tiles = (a.r + 15) / 16;
#pragma unroll 1
    for (int jt = j0 / 16; jt < min(j0 / 16 + RT, tiles); ++jt) {
        v4f first[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) first[c] = v4f{0, 0, 0, 0};
#pragma unroll 1
        for (int row = it.row0; row < it.row1; row += kRows) {
            int token[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) token[i] = token_of(a.row_token[row + kg * 8 + i], a.T);
            Wide x;
            x.load(w, token, col, in);
            x.settle();
            const v4u p = w.p[((int64_t)(row >> 5) * tiles + jt) * kOuterParts * 64 + lane];
#pragma unroll
            for (int c = 0; c < 8; ++c) first[c] = mfma(p, x.column(c), first[c]);
        }
        const int rank = jt * 16 + kg * 4;
        if (!in || rank >= a.r) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *o = out + (SECOND ? (int64_t)(col + c) * a.r + rank + i : (int64_t)(rank + i) * w.C + col + c);
                if (*o != *o) *o = first[c][i];
            }
    }
}

// One block: an item's rows, 128 columns of a wide matrix, RT tiles of 16
// ranks.  A lane loads 8 columns of 8 rows and turns them into eight fragments
// with one permutation for every two values, so nothing is staged.  Its waves
// take blocks of 32 rows in turn.  8192 rows of rank 32, x [4096] in 8 bits and d_y
// [6144]: 35 to 40 us (134 MB, 3.4 TB/s), half of it vector arithmetic on the
// values' forms; 4001 rows of rank 16, 2048 and 1536 in bf16: 12.8 us.  x's form
// changes little: whole gradients at rank 32 take 104.5 us with x in bf16, 104.7
// canonical and 105.1 packed, at rank 128 206, 207 and 210.
template <int RT, class Wide, bool SECOND>
__device__ __forceinline__ void outer_block(const LoraOuter &a, const Item &it, int slab, int j0, int lane, int wave,
                                            v4u (&red)[2][RT * 8][64]) {
    const LoraWide &w = a.wide[SECOND ? 1 : 0];
    const int m = lane & 15, kg = lane >> 4;
    const int col = slab * 128 + m * 8;
    const bool in = col < w.C;
    v4f acc[RT][8];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = v4f{0, 0, 0, 0};
    outer_rows<RT, Wide>(a, w, it, j0 / 16, col, in, lane, wave, acc);

    // the four waves' sums, always in the same order: (0 + 2) + (1 + 3)
    if (wave >= 2) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) red[wave - 2][i][lane] = __builtin_bit_cast(v4u, acc[i >> 3][i & 7]);
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) acc[i >> 3][i & 7] += __builtin_bit_cast(v4f, red[wave][i][lane]);
    }
    __syncthreads();
    if (wave == 1) {
#pragma unroll
        for (int i = 0; i < RT * 8; ++i) red[0][i][lane] = __builtin_bit_cast(v4u, acc[i >> 3][i & 7]);
    }
    __syncthreads();
    if (wave != 0) return;
    const int64_t size = (int64_t)a.r * w.C;
    float *out = it.slot < 0 ? w.out + it.e * size : w.part + it.slot * size;
    bool lost = false;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int rank = j0 + j * 16 + kg * 4;           // four ranks, eight columns
        if (!in || rank >= a.r) continue;
        v4f v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = acc[j][c] + __builtin_bit_cast(v4f, red[0][j * 8 + c][lane]);
        lost = lost || has_nan(v);
        if constexpr (SECOND) {                          // [C][r]
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
    if (__builtin_expect(__ballot(lost) != 0, 0)) outer_first<RT, Wide, SECOND>(a, w, it, j0, col, in, lane, out);
}

template <int RT, class WideX>
__global__ __launch_bounds__(kBlock, RT <= 2 ? 2 : 1) void lora_outer_kernel(const LoraOuter a) {
    __shared__ v4u red[2][RT * 8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = a.wide[0].slabs + a.wide[1].slabs;
    int at = blockIdx.x % (per * a.passes);
    const Item it = item_of(a, blockIdx.x / (per * a.passes), lane);
    if (it.e < 0 || it.slot >= a.slots) return;          // the whole block
    const int j0 = at / per * RT * 16;
    at %= per;
    if (at >= a.wide[0].slabs) outer_block<RT, WideBf16, true>(a, it, at - a.wide[0].slabs, j0, lane, wave, red);
    else outer_block<RT, WideX, false>(a, it, at, j0, lane, wave, red);
}

// The sums of adapters with several items, slots in order; block row y is the
// y-th such adapter.  4 to 5 us.
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
    m = min(m, a.slots - slot);
    v4f v = {0, 0, 0, 0};
    for (int n0 = 0; n0 < m; n0 += 8) {                  // eight in flight
        v4f part[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) part[n] = *reinterpret_cast<const v4f *>(p + (n0 + n < m ? n0 + n : 0) * size);
#pragma unroll
        for (int n = 0; n < 8; ++n)
            if (n0 + n < m) v += part[n];
    }
    *reinterpret_cast<v4f *>(w.out + e * size + at) = v;
}

template <class Y, int KT>
void start_expand(LoraExpand a, int cus, hipStream_t stream) {
    // Blocks of 64 rows (32 where y is fp32) that go through several columns each, as many as are resident at once (by
    // their registers two a compute unit, one for ranks above 64), where there are that many columns; else of 32 rows
    // and 256 columns (8192 rows of rank 64 to 6144 so 60 us for 51).
    constexpr int kWide = sizeof(Y) == 4 ? 1 : 2, kResident = KT == 4 ? 1 : 2;
    const int64_t blocks = a.rows / kRows, groups = ceil_div(blocks, kWide), tiles = a.N ? ceil_div(a.N, 256) : 1;
    if (groups * tiles >= 2 * kResident * cus) {
        const int64_t step = kResident * cus / groups;
        a.step = (int)(step > 1 ? step : 1);
        lora_expand_kernel<Y, KT, kWide, true><<<(unsigned)(groups * a.step), kBlock, 0, stream>>>(a);
    } else {
        a.step = (int)tiles;
        lora_expand_kernel<Y, KT, 1, false><<<(unsigned)(blocks * tiles), kBlock, 0, stream>>>(a);
    }
}
template <class Y>
void start_expand(const LoraExpand &a, int cus, hipStream_t stream) {
    if (a.r <= 32) start_expand<Y, 1>(a, cus, stream);
    else if (a.r <= 64) start_expand<Y, 2>(a, cus, stream);
    else start_expand<Y, 4>(a, cus, stream);
}
template <class Y>
void start_both(const LoraShrink &s, const LoraExpand &a, unsigned grid, hipStream_t stream) {
    if (a.r <= 16) lora_both_kernel<Y, 1><<<grid, kBothWaves * 64, 0, stream>>>(s, a);
    else if (a.r <= 32) lora_both_kernel<Y, 2><<<grid, kBothWaves * 64, 0, stream>>>(s, a);
    else lora_both_kernel<Y, 4><<<grid, kBothWaves * 64, 0, stream>>>(s, a);
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
    // give every wave of a block a chunk (one row of 12288, rank 16: 15.4 us whole, 10.6 cut, the launch of both products
    // in it)
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
    const int cus = device_cu_count();
    if (y_bf16) start_expand<uint16_t>(a, cus, stream);
    else start_expand<float>(a, cus, stream);
    return hipGetLastError();
}

// One launch instead of two.  Where there is a block of rows for more than every
// second CU, no block takes what another one takes too (7936 rows of rank 64,
// 4096 to 6144: 51.3 us for 61.1; 4320 rows, 135 blocks, at worst 52.5 for 49.3 with
// 12288 columns of x, but 120 for 77 with 32768, which few blocks read too slowly:
// there from two of three CUs on, 182 blocks 135 for 146), up to the padding of a batch that fills
// the CUs once (8192 rows of 8 adapters, 263 blocks: 56.7 for 64.6; at 391 blocks
// 95.7 for 94.8, with 12288 columns 165 for 145).  With fewer blocks, where a
// block's rows of x and A are short enough that taking them several times costs
// less than the second launch (one row of rank 16, 4096 to 6144: 10.4 us for 13.2
// with the host's part, 64 rows of as many adapters 13.1 for 13.5; past the bound
// 512 rows of 8 adapters take 15.2 for 13.0, one row of 12288 columns 15.4 for 13.1).
bool lora_both(int64_t rows, int64_t T, int64_t r, int64_t K, int cus) {
    const int64_t blocks = rows / kRows, most = 96 * 1024;
    if (r > 64 || blocks > cus + cus / 16) return false;
    const int64_t used = ceil_div(T, blocks);
    if (blocks > (K <= 16384 ? cus / 2 : cus * 2 / 3)) return true;
    return K <= most && K * ((used < kRows ? used : kRows) + r) <= most;
}

hipError_t launch_lora_both(const LoraShrink &s, LoraExpand a, bool y_bf16, hipStream_t stream) {
    const int64_t blocks = a.rows / kRows, tiles = a.N ? ceil_div(a.N, kBothWaves * 64) : 1;
    const int64_t step = device_cu_count() / blocks;
    a.step = (int)(step < 1 ? 1 : step < tiles ? step : tiles);
    if (y_bf16) start_both<uint16_t>(s, a, (unsigned)(blocks * a.step), stream);
    else start_both<float>(s, a, (unsigned)(blocks * a.step), stream);
    return hipGetLastError();
}

hipError_t launch_lora_prepare(const LoraPrepare &a, hipStream_t stream) {
    int64_t most = ceil_div(a.rows / kRows * ceil_div(a.r, 16), kWaves);
    for (const LoraPrepare::Job &j : a.job) {
        const int64_t n = a.E * ceil_div(j.P, 64) * ceil_div(j.Q, 64);
        most = most > n ? most : n;
    }
    const int64_t cap = 8 * (int64_t)device_cu_count();
    lora_prepare_kernel<<<dim3((unsigned)(most < cap ? most : cap), 3), kBlock, 0, stream>>>(a);
    return hipGetLastError();
}

LoraOuterPlan lora_outer_plan(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N, int cus) {
    const int64_t passes = ceil_div(r, 64), slabs = (ceil_div(K, 128) + ceil_div(N, 128)) * passes;
    const int64_t wanted = slabs < 2 * cus ? 2 * cus / slabs : 1;
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
