// Host-side launchers of the gfx950 MXFP8 kernels (internal to the library;
// the public C ABI is include/mxfp8.h).  Every launcher assumes its
// arguments were validated by the API layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Compute units of the current device (cached per device).
int device_cu_count();

// Dense GEMM tiling: big_cols tile columns of 256x256 tiles over the leading
// columns, then small_cols tile columns of 256x128 tiles (either may be 0).
struct DenseTiling {
    int big_cols, small_cols;
};
DenseTiling dense_tiling(int64_t M, int64_t N, int cus);

// Split-K plan of a dense GEMM: K slices of split_steps k-steps, fp32
// partials of splits * M * N floats (splits == 1: no split).
struct SplitPlan {
    int splits, split_steps;
    int64_t workspace_bytes;
};
SplitPlan splitk_plan(int64_t M, int64_t N, int64_t K, int cus);
// partial tiles into `workspace`, then C = their sum (slice order)
// mxfp8_gemm_accurate: BF16 MFMA on exactly converted operands
hipError_t launch_gemm_accurate(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                                const uint8_t *b_s, bool b_packed, int64_t M, int64_t N, int64_t K, void *c,
                                bool c_bf16, hipStream_t stream);
// device address and size of the static split-K scratch on the current device
hipError_t splitk_scratch(void **ptr, size_t *bytes);
hipError_t launch_gemm_splitk(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q, const uint8_t *b_s,
                              bool b_packed, int64_t M, int64_t N, int64_t K, void *c, bool c_bf16,
                              const SplitPlan &plan, float *workspace, hipStream_t stream);

hipError_t launch_quantize(const uint16_t *x, int64_t rows, int64_t cols, int axis, uint8_t *q,
                           uint8_t *scales, hipStream_t stream);

// x[batch][rows][cols] -> q[batch][cols][rows], scales[batch][cols][rows/32]
hipError_t launch_quantize_axis0_batched(const uint16_t *x, int64_t batch, int64_t rows,
                                         int64_t cols, uint8_t *q, uint8_t *scales,
                                         hipStream_t stream);

// axis-1 quantize of rows x[idx[i]] (zero rows for indices outside [0, rows_in))
hipError_t launch_quantize_gather(const uint16_t *x, int64_t rows_in, int64_t cols,
                                  const int64_t *idx, int64_t rows_out, uint8_t *q,
                                  uint8_t *scales, hipStream_t stream);

hipError_t launch_quantize_dual(const uint16_t *x, int64_t rows, int64_t cols, uint8_t *q_row,
                                uint8_t *s_row, uint8_t *q_col, uint8_t *s_col, hipStream_t stream);
hipError_t launch_quantize_gather_packed(const uint16_t *x, int64_t rows_in, int64_t cols, const int64_t *idx,
                                         int64_t rows_out, uint8_t *q_packed, uint8_t *s_packed, hipStream_t stream);
hipError_t launch_quantize_dual_grouped_packed(const uint16_t *x, int64_t rows, int64_t cols, uint8_t *qr_packed,
                                               uint8_t *sr_packed, uint8_t *qc, uint8_t *sc, bool col_packed,
                                               const int32_t *src_off, const int32_t *dst_off, int64_t G,
                                               int64_t rows_out, hipStream_t stream);
hipError_t launch_grouped_gemm_wgrad_packed(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                                            const uint8_t *b_s, const int32_t *offsets, int64_t G, int64_t T,
                                            int64_t M, int64_t N, void *c, bool c_bf16, hipStream_t stream);
hipError_t launch_quantize_dual_packed(const uint16_t *x, int64_t batch, int64_t rows, int64_t cols,
                                       uint8_t *qr_packed, uint8_t *sr_packed, uint8_t *qc_packed,
                                       uint8_t *sc_packed, hipStream_t stream);

// axis 1 (q_row / s_row may be null) and axis 0 regrouped by token offsets
// into q_col[cols][rows_out], s_col[cols][rows_out/32], pads zeroed
hipError_t launch_quantize_dual_grouped(const uint16_t *x, int64_t rows, int64_t cols, uint8_t *q_row,
                                        uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                                        const int32_t *src_off, const int32_t *dst_off, int64_t G,
                                        int64_t rows_out, hipStream_t stream);

// x[batch][rows][cols] along axis 0 into the packed layout of the transposed
// grid (what repack writes for q[batch][cols][rows]); rows % 32 == 0,
// cols % 8 == 0
hipError_t launch_quantize_axis0_packed(const uint16_t *x, int64_t batch, int64_t rows, int64_t cols,
                                        uint8_t *q_packed, uint8_t *s_packed, hipStream_t stream);

// Several tensors quantized along axis 1 in one launch.  Tensor i has
// nblocks[i] = rows * cols / 32 blocks and ceil(nblocks[i] / 64) wave-steps,
// which are steps step_end[i-1] .. step_end[i]-1 of the launch.
constexpr int kQuantJobsMax = 8;
struct QuantJobs {
    const uint16_t *x[kQuantJobsMax];
    uint8_t *q[kQuantJobsMax];
    uint8_t *s[kQuantJobsMax];
    int64_t nblocks[kQuantJobsMax];
    int64_t step_end[kQuantJobsMax];
    // packed[i]: q/s of job i are the packed layout of its grid; its steps are
    // (16-row atom, k-step) pairs over ceil(rows / 256) * 16 atoms
    int64_t rows[kQuantJobsMax];
    int64_t cols[kQuantJobsMax];
    int32_t packed[kQuantJobsMax];
    int count;
};
hipError_t launch_quantize_many(const QuantJobs &jobs, hipStream_t stream);

// A list of weights quantized into the packed layout in one launch.  Weight i
// is BF16 [batch_i][N[i]][K[i]]; its tiles are tile_end[i-1] .. tile_end[i]-1
// of the launch (tile_end[i] - tile_end[i-1] = batch_i * panels * k-steps).
constexpr int kPackedJobsMax = 32;
struct PackedJobs {
    const uint16_t *w[kPackedJobsMax];
    uint8_t *qc[kPackedJobsMax];      // canonical q, or null
    uint8_t *sc[kPackedJobsMax];      // canonical scales, or null
    uint8_t *qp[kPackedJobsMax];
    uint32_t *sp[kPackedJobsMax];
    int64_t N[kPackedJobsMax];
    int64_t K[kPackedJobsMax];
    int64_t tile_end[kPackedJobsMax];
    int count;
};
hipError_t launch_quantize_packed_jobs(const PackedJobs &jobs, hipStream_t stream);

// q / scales may be null (packed output only)
hipError_t launch_quantize_packed(const uint16_t *w, int64_t batch, int64_t N, int64_t K,
                                  uint8_t *q, uint8_t *scales, uint8_t *q_packed,
                                  uint8_t *s_packed, hipStream_t stream);

hipError_t launch_dequantize(const uint8_t *q, const uint8_t *scales, int64_t rows, int64_t cols,
                             int axis, void *out, bool out_bf16, hipStream_t stream);

hipError_t launch_repack(const uint8_t *q, const uint8_t *scales, int64_t batch, int64_t N,
                         int64_t K, uint8_t *q_packed, uint8_t *s_packed, hipStream_t stream);

// the tiles launch_gemm_packed takes: gemm_ws_kernel's 256x128 or 128x128
// tiles, or launch_gemm's tilings
enum class PackedTiling { kWs, kWsHalf, kDense };
PackedTiling packed_tiling(int64_t M, int64_t N, bool c_bf16, int cus);
hipError_t launch_gemm_packed(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q, const uint8_t *b_s,
                              int64_t M, int64_t N, int64_t K, void *c, bool c_bf16, hipStream_t stream);
hipError_t launch_gemm_packed_splitk(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                                     const uint8_t *b_s, int64_t M, int64_t N, int64_t K, void *c,
                                     bool c_bf16, const SplitPlan &sp, float *workspace, hipStream_t stream);
hipError_t launch_grouped_gemm_packed(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                                      const uint8_t *b_s, const int32_t *offsets, int64_t G, int64_t M_total,
                                      int64_t N, int64_t K, void *c, bool c_bf16, hipStream_t stream);
hipError_t launch_gemm(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                       const uint8_t *b_s, bool b_packed, int64_t M, int64_t N, int64_t K, void *c,
                       bool c_bf16, hipStream_t stream);

hipError_t launch_grouped_gemm(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                               const uint8_t *b_s, const int32_t *offsets, int64_t G,
                               int64_t M_total, int64_t N, int64_t K, void *c, bool c_bf16,
                               hipStream_t stream);

// Self-check workspace: byte offsets of its parts (256-byte aligned) and the
// total size, for a probe of M rows against weights [N][K].
struct SelfcheckWorkspace {
    int64_t xq, xs, y, yref, part, total;
};
SelfcheckWorkspace selfcheck_workspace(int64_t M, int64_t N, int64_t K);

// Reference Y_ref = X * dequant(W)^T in fp32 (X bf16 [M][K], W canonical [N][K]).
hipError_t launch_selfcheck_ref(const uint16_t *x, int64_t M, int64_t N, int64_t K,
                                const uint8_t *wq, const uint8_t *ws, float *yref,
                                hipStream_t stream);

// out[0] = ||y - yref|| / ||yref|| (NaN if not finite), out[1..2] the sums.
hipError_t launch_selfcheck_error(const float *y, const float *yref, int64_t n, double *part,
                                  double *out, hipStream_t stream);

// C[g] = A[:, o_g:o_g+1] B[:, o_g:o_g+1]^T, A [M][T], B [N][T] canonical (row stride T)
hipError_t launch_grouped_gemm_wgrad(const uint8_t *a_q, const uint8_t *a_s, const uint8_t *b_q,
                                     const uint8_t *b_s, const int32_t *offsets, int64_t G,
                                     int64_t T, int64_t M, int64_t N, void *c, bool c_bf16,
                                     hipStream_t stream);

// Expert routing (route.hip).  T >= 1 rows of E logits, ld elements apart.
constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxGroups = 64;
struct RouteArgs {
    const void *x;              // logits [T][ld]
    int64_t ld, T;
    const float *bias;          // [E] or null
    int32_t *ids;               // [T][k] (read by the backward)
    float *w;                   // [T][k]
    const float *dw;            // [T][k], backward only
    void *dx;                   // [T][E], backward only
    float scale;
    int E, k, groups, size, kept, group_top;   // size = E / groups
    bool sigmoid, renorm;
    // set by the launchers
    bool order_x, order_exact;
    int lanes_shift, candidates;
};
hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs &a, bool bf16, hipStream_t stream);

// Row tables (tables.hip).  pairs >= 1; hist: chunks * E ints where a counting
// launch comes first (route_tables_workspace_bytes is not 0).
constexpr int kTablesMaxExperts = 1024;
constexpr int kTablesMaxChunks = 64;
struct RouteTables {
    const int32_t *ids;         // [pairs]
    int32_t *offsets, *counts, *pair_row, *hist;
    int64_t *row_token;         // [rows]
    int64_t pairs, rows;
    int k, E, pad;
    // set by the launcher
    int64_t chunk;
    int chunks, id_bits, width;
};
int64_t route_tables_workspace_bytes(int64_t pairs, int64_t E);
hipError_t launch_route_tables(RouteTables a, hipStream_t stream);

// Expert rows back to tokens (combine.hip)
struct CombineArgs {
    const void *y;              // [rows][H]
    const int32_t *pair_row;    // [T][k]
    const float *w;             // [T][k]
    void *out;                  // [T][H]
    const void *d_out;          // [T][H], backward only
    const int64_t *row_token;   // [rows], backward only
    void *d_y;                  // [rows][H], backward only
    float *d_w;                 // [T][k], backward only
    int64_t T, rows, H;
    int k;
};
hipError_t launch_combine(const CombineArgs &a, bool bf16, hipStream_t stream);
hipError_t launch_combine_backward(const CombineArgs &a, bool bf16, hipStream_t stream);

// Token log-probabilities (logprobs.hip)
constexpr int kLogprobsMaxTop = 64;
struct LogprobsArgs {
    const void *x;              // logits [T][ld]
    int64_t ld, T, V;
    const int64_t *targets;     // [T]
    double temperature;
    int top;
    float *logprobs, *entropy, *stats;      // [T], [T], [T][2]; read by the backward (entropy, stats)
    float *top_logprobs;                    // [T][top]
    int64_t *top_ids;                       // [T][top]
    void *workspace;
    const float *d_logprobs, *d_entropy;    // [T], either may be null
    void *dx;                               // [T][ld_out]
    int64_t ld_out;
    // set by the launcher
    double inv_temperature;
    float scale, inv, inv_low;              // log2(e) / temperature; 1 / temperature in two parts
    int64_t slice;
    int slices;
};
int64_t logprobs_workspace_bytes(int64_t T, int64_t V, int top, int cus);
hipError_t launch_logprobs(LogprobsArgs a, bool bf16, size_t workspace_bytes, hipStream_t stream);
hipError_t launch_logprobs_backward(LogprobsArgs a, bool bf16, hipStream_t stream);

// Gated activation with an 8-bit checkpoint (swiglu.hip).  T >= 1.
struct SwigluArgs {
    const uint16_t *x;          // gu [T][ld], or d_h [T][ld] (backward)
    int64_t ld, T;
    int I;
    uint16_t *h;                // [T][I] or null
    uint8_t *hq, *hs;           // h's grid, or null
    uint8_t *q, *s;             // the checkpoint [T][2 I], [T][2 I / 32] (forward: or null)
    uint16_t *dx;               // d_gu [T][2 I], backward only
};
hipError_t launch_swiglu(const SwigluArgs &a, bool h_packed, hipStream_t stream);
hipError_t launch_swiglu_backward(const SwigluArgs &a, hipStream_t stream);

// Low-rank adapters (lora.hip).  rows: sorted rows, a multiple of 32.
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 1024;
typedef uint32_t LoraVec __attribute__((ext_vector_type(4)));
struct LoraShrink {
    const uint16_t *x;          // [T][ld], K columns
    int64_t ld, T;
    const uint16_t *w;          // [E][r][K]
    const int32_t *offsets;     // [E + 1]
    const int64_t *row_token;   // [rows]
    int64_t rows;
    float *part;                // [splits][rows][r]
    int E, r, K, splits, slice;
};
struct LoraCut {
    int splits, slice;
};
LoraCut lora_cut(int64_t rows, int64_t K, int cus);
hipError_t launch_lora_shrink(const LoraShrink &a, hipStream_t stream);
struct LoraExpand {
    void *y;                    // [T][ld], N columns
    int64_t ld, T;
    const uint16_t *w;          // [E][N][r]
    const float *scales;        // [E] or null
    const int32_t *offsets;
    const int64_t *row_token;
    int64_t rows;
    const float *part;          // [splits][rows][r]
    float *hidden;              // [rows][r] or null: the sum of the partials
    LoraVec *packed;      // or null: lora_packed_bytes of it, scaled
    int E, r, N, splits;        // N = 0: hidden alone
    int step;                   // set by the launcher: blocks beside each other on the same rows
};
hipError_t launch_lora_expand(LoraExpand a, bool y_bf16, hipStream_t stream);
// both in one launch, without partials, where lora_both says so
bool lora_both(int64_t rows, int64_t T, int64_t r, int64_t K, int cus);
hipError_t launch_lora_both(const LoraShrink &s, LoraExpand a, bool y_bf16, hipStream_t stream);
struct LoraPrepare {
    struct Job {
        const uint16_t *from;   // [E][P][Q]
        uint16_t *to;           // [E][Q][P]
        int P, Q;
    } job[2];
    const float *hidden;        // [rows][r]
    LoraVec *packed;      // lora_packed_bytes of it, scaled
    const float *scales;
    const int32_t *offsets;
    const int64_t *row_token;
    int64_t rows, T;
    int E, r;
};
// rows of P as the outer products take them
inline int64_t lora_packed_bytes(int64_t rows, int64_t r) { return rows / 32 * ((r + 15) / 16) * 3 * 1024; }
hipError_t launch_lora_prepare(const LoraPrepare &a, hipStream_t stream);
// sums over rows, cut into chunks: items at most, slots of partial sums at most
struct LoraOuterPlan {
    int64_t chunk, items, slots;
};
LoraOuterPlan lora_outer_plan(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N, int cus);
struct LoraWide {
    const LoraVec *p;     // lora_packed_bytes
    const void *x;              // [T][ld] bf16, or a grid's codes
    const uint8_t *s;           // the grid's scales
    int64_t ld, ksteps;
    int C;                      // columns
    float *out;                 // [E][r][C] (the first) or [E][C][r] (the second)
    float *part;                // slots of the same
    int slabs;                  // set by the launcher
};
struct LoraOuter {
    LoraWide wide[2];           // the second is bf16
    const int32_t *offsets;
    const int64_t *row_token;
    int64_t rows, T;
    int E, r;
    int chunk, slots, passes;   // set by the launcher
};
// form of the first wide matrix: 0 bf16, 1 canonical grid, 2 packed
hipError_t launch_lora_outer(LoraOuter a, const LoraOuterPlan &plan, int form, hipStream_t stream);

// Verification of drafted tokens (drafts.hip).  B >= 1.
struct DraftArgs {
    const void *x;              // the target's logits [R][ld]
    int64_t ld, R, V, B;
    const int32_t *offsets;     // [B + 1]
    const int64_t *ids;         // [R - B]
    const float *u;             // [R - B]
    const void *d;              // the draft's logits [R - B][ld_d] or null
    int64_t ld_d;
    const float *noise;         // [B][ld_n]
    int64_t ld_n;
    double temperature;
    int32_t *accepted;          // [B]
    int64_t *tokens;            // [R]
    float *logprobs;            // [R]
    void *workspace;
    int64_t rows;               // R, and with the draft's logits R - B more
    // set by the launcher
    double inv_temperature, scale64;        // 1 / temperature, log2(e) / temperature
    float scale;
    int64_t slice, cut;
    int slices, cuts;
};
// slices of a row's sums, cuts of a request's race, their lengths, and the workspace they take
struct DraftCut {
    int slices, cuts;
    int64_t slice, cut, bytes;
};
DraftCut draft_cut(int64_t rows, int64_t B, int64_t V, int cus);
hipError_t launch_drafts(DraftArgs a, bool bf16, hipStream_t stream);

// Packed weight layout geometry (see mxfp8_repack in include/mxfp8.h).
constexpr int64_t kPanelRows = 256;   // rows per packed panel
constexpr int64_t kKStep = 128;       // K bytes per packed k-step (one MFMA K)
constexpr int64_t kTileBytes = kPanelRows * kKStep;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t packed_panels(int64_t N) { return ceil_div(N, kPanelRows); }
inline int64_t packed_ksteps(int64_t K) { return ceil_div(K, kKStep); }
inline int64_t packed_q_bytes(int64_t batch, int64_t N, int64_t K) {
    return batch * packed_panels(N) * packed_ksteps(K) * kTileBytes;
}
// scales: [batch][panel][k-step][16 atoms of 16 rows][64 lanes] bytes
constexpr int64_t kScaleStepBytes = 16 * 64;
inline int64_t packed_s_bytes(int64_t batch, int64_t N, int64_t K) {
    return batch * packed_panels(N) * packed_ksteps(K) * kScaleStepBytes;
}

}  // namespace mx
