// The expert-sorted row tables of a routed batch.
#include "mx_launch.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

constexpr int kThreads = 512;
constexpr int kWavesT = kThreads / 64;
constexpr int kCounts = 16;        // chunk counts of a thread in flight
constexpr int kAlone = 8;          // most chunks without a counting pass of their own; ids of a thread in flight

__device__ __forceinline__ bool real_expert(int id, int E) { return (unsigned)id < (unsigned)E; }

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// Sum of the lanes up to and with one's own.  Inside a row of 16 and from row
// to row the steps are lane shifts of the vector ALU; lanes that none reaches
// add 0.
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp_add<0x111, 0xF>(v);                    // row_shr:1
    v += dpp_add<0x112, 0xF>(v);                    // row_shr:2
    v += dpp_add<0x114, 0xF>(v);                    // row_shr:4
    v += dpp_add<0x118, 0xF>(v);                    // row_shr:8
    v += dpp_add<0x142, 0xA>(v);                    // row_bcast:15 into rows 1 and 3
    v += dpp_add<0x143, 0xC>(v);                    // row_bcast:31 into rows 2 and 3
    return v;
}

// counts of the experts in one chunk of pairs -> hist[chunk][E]
__global__ __launch_bounds__(kThreads) void route_count_kernel(const RouteTables a) {
    __shared__ int cnt[kTablesMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.chunk;
    const int64_t hi = lo + a.chunk < a.pairs ? lo + a.chunk : a.pairs;
    for (int64_t p = lo + threadIdx.x; p < hi; p += kThreads) {
        const int id = a.ids[p];
        if (real_expert(id, a.E)) atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

// Places a chunk's pairs: row = start of the expert's padded group + pairs of
// that expert in earlier chunks, earlier waves of the chunk, and earlier in
// the wave, so rows come in (expert, pair) order whatever runs first.  The
// rank inside a wave is the count of lower lanes with the same expert, found
// with one ballot per bit of the id.  Without a table of the chunks' counts
// (hist null: few chunks) a block counts all pairs itself: 2048 pairs over 256
// experts 6.8 us against 9.6 us with the counting launch before it, and that
// launch and its workspace cost the caller another 5 us.
//
// Latency-bound: a chain of loads, LDS counts and barriers (256 pairs over 128
// experts 5.7 us; 131072 pairs over 256 experts 3.0 us of counting and 9.1 us
// here, where their bytes would take 0.4 us).  The chunk counts are summed by
// several threads an expert with their loads in flight: one thread an expert
// took 28.2 us.  Scans over lane shifts and padding rows by half waves save
// 1.1 us of the chain.
__global__ __launch_bounds__(kThreads) void route_place_kernel(const RouteTables a) {
    __shared__ int start[kTablesMaxExperts + 1];     // padded group starts
    __shared__ int total[kTablesMaxExperts];
    __shared__ int ahead[kTablesMaxExperts];         // hist null: pairs in earlier chunks
    __shared__ int at[kWavesT][kTablesMaxExperts];   // next row of (wave, expert)
    __shared__ int sums[kWavesT];
    __shared__ int2 joined[kThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.E; e += kThreads)
#pragma unroll
        for (int w = 0; w < kWavesT; ++w) at[w][e] = 0;
    if (!a.hist)
        for (int e = tid; e < a.E; e += kThreads) ahead[e] = total[e] = 0;    // pairs of the chunks before, after
    __syncthreads();

    const int64_t lo = (int64_t)blockIdx.x * a.chunk;
    const int64_t hi = lo + a.chunk < a.pairs ? lo + a.chunk : a.pairs;
    const int64_t per = a.chunk / kWavesT;           // pairs of a wave, a multiple of 64
    const int64_t wlo = lo + wave * per;
    const int64_t whi = wlo + per < hi ? wlo + per : hi;
#pragma unroll 4
    for (int64_t p = wlo + lane; p < whi; p += 64) {
        const int id = a.ids[p];
        if (real_expert(id, a.E)) atomicAdd(&at[wave][id], 1);
    }
    if (!a.hist && a.chunks > 1) {
        for (int64_t p0 = 0; p0 < a.pairs; p0 += kAlone * kThreads) {
            int id[kAlone];
#pragma unroll
            for (int u = 0; u < kAlone; ++u) {
                const int64_t p = p0 + u * kThreads + tid;
                id[u] = p < a.pairs && (p < lo || p >= hi) ? a.ids[p] : -1;
            }
#pragma unroll
            for (int u = 0; u < kAlone; ++u)
                if (real_expert(id[u], a.E)) atomicAdd(p0 + u * kThreads + tid < lo ? &ahead[id[u]] : &total[id[u]], 1);
        }
    }
    __syncthreads();

    // pairs of every expert in all chunks and in the chunks before this one:
    // `parts` threads an expert, each with every parts-th chunk
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + (tid & (a.width - 1)), part = tid / a.width;
        int all = 0, before = 0;
        if (e < a.E) {
            if (!a.hist) {
                if (part == 0) {
                    for (int w = 0; w < kWavesT; ++w) all += at[w][e];
                    before = ahead[e];
                    all += before + total[e];
                }
            } else {
                const int step = kThreads / a.width;
                for (int c0 = part; c0 < a.chunks; c0 += kCounts * step) {
                    int n[kCounts];
#pragma unroll
                    for (int u = 0; u < kCounts; ++u) {
                        const int c = c0 + u * step;
                        n[u] = a.hist[(int64_t)(c < a.chunks ? c : part) * a.E + e];
                    }
#pragma unroll
                    for (int u = 0; u < kCounts; ++u) {
                        const int c = c0 + u * step;
                        before += c < (int)blockIdx.x ? n[u] : 0;
                        all += c < a.chunks ? n[u] : 0;
                    }
                }
            }
        }
        joined[tid] = make_int2(all, before);
        __syncthreads();
        all = before = 0;
        if (tid < a.width && e < a.E) {
            for (int q = tid; q < kThreads; q += a.width) {
                all += joined[q].x;
                before += joined[q].y;
            }
            total[e] = all;
        }
        // exclusive scan of the padded totals over the experts
        const int padded = (all + a.pad - 1) / a.pad * a.pad;
        const int scan = wave_scan(padded);
        if (lane == 63) sums[wave] = scan;
        __syncthreads();
        int first = scan - padded + (e0 ? start[e0] : 0);
        for (int w = 0; w < wave; ++w) first += sums[w];
        if (tid < a.width && e < a.E) {
            start[e] = first;
            start[e + 1] = first + padded;       // the next expert's own start, and the end after the last
            int next = first + before;
#pragma unroll
            for (int w = 0; w < kWavesT; ++w) {
                const int n = at[w][e];
                at[w][e] = next;
                next += n;
            }
        }
        __syncthreads();
    }

    int ahead_id = wlo + lane < whi ? a.ids[wlo + lane] : -1;
    for (int64_t base = wlo; base < whi; base += 64) {
        const int64_t p = base + lane;
        const int id = ahead_id;
        ahead_id = p + 64 < whi ? a.ids[p + 64] : -1;
        const bool real = real_expert(id, a.E);
        uint64_t same = __ballot(real);
        for (int b = 0; b < a.id_bits; ++b) {
            const uint64_t m = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? m : ~m;
        }
        const uint64_t lower = same & ((1ull << lane) - 1);
        const int rank = __builtin_popcountll(lower);
        int row = -1;
        if (real) row = at[wave][id] + rank;
        wave_sync();
        if (real && (same >> lane) == 1ull) at[wave][id] = row + 1;   // highest lane of its expert
        wave_sync();
        if (p < whi) {
            a.pair_row[p] = row;
            if (real) a.row_token[row] = (uint32_t)p / (uint32_t)a.k;
        }
    }

    // padding rows, the rows past the last group, and the tables of the groups
#pragma unroll 4
    for (int e = blockIdx.x * (kThreads / 32) + tid / 32; e < a.E; e += gridDim.x * (kThreads / 32))
        for (int r = start[e] + total[e] + (tid & 31); r < start[e + 1]; r += 32) a.row_token[r] = -1;
    for (int64_t r = start[a.E] + (int64_t)blockIdx.x * kThreads + tid; r < a.rows; r += (int64_t)gridDim.x * kThreads)
        a.row_token[r] = -1;
    if (blockIdx.x == 0) {
        for (int e = tid; e <= a.E; e += kThreads) a.offsets[e] = start[e];
        for (int e = tid; e < a.E; e += kThreads) a.counts[e] = total[e];
    }
}

}  // namespace

// Chunks of pairs, one block each: one chunk while a block can place them in
// a few steps, then at most kTablesMaxChunks.
static int64_t route_tables_chunk(int64_t pairs) {
    int64_t chunk = 2 * kThreads;
    if (ceil_div(pairs, chunk) > kTablesMaxChunks) chunk = ceil_div(ceil_div(pairs, kTablesMaxChunks), kThreads) * kThreads;
    return chunk;
}

int64_t route_tables_workspace_bytes(int64_t pairs, int64_t E) {
    const int64_t chunks = ceil_div(pairs, route_tables_chunk(pairs));
    return chunks > kAlone ? chunks * E * 4 : 0;
}

hipError_t launch_route_tables(RouteTables a, hipStream_t stream) {
    a.chunk = route_tables_chunk(a.pairs);
    a.chunks = (int)ceil_div(a.pairs, a.chunk);
    a.id_bits = 0;
    while ((1 << a.id_bits) < a.E) ++a.id_bits;
    a.width = 64;
    while (a.width < a.E && a.width < kThreads) a.width <<= 1;
    if (a.chunks <= kAlone) a.hist = nullptr;
    if (a.hist) route_count_kernel<<<(unsigned)a.chunks, kThreads, 0, stream>>>(a);
    route_place_kernel<<<(unsigned)a.chunks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace mx
