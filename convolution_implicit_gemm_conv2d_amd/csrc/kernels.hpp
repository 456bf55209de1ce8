// Launchers of the HIP kernels (host side).  Each returns hipSuccess or the
// launch error; arguments were validated by the caller.
#pragma once

#include "common.hpp"

namespace convmi {

// Compute units of the current device (queried once per device).
int device_cu_count();

// Records the message of a failed call on this thread; returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Generic direct forward, any geometry, layout and dtype (dtype 0 fp32, 1 bf16).
hipError_t launch_fwd_direct(const void* x, const void* w, const void* bias, void* y,
                             const Geom& g, int dtype, hipStream_t s);
// Generic input gradient as a per-element gather, plus a per-channel bias
// (NULL for none; the transposed convolution has one).
hipError_t launch_dx_gather(const void* dy, const void* w, const void* bias, void* dx,
                            const Geom& g, int dtype, hipStream_t s);

// Fast paths.  Each has a predicate (can_*) that the dispatcher checks first.
bool can_pointwise(const Geom& g, int dtype);
hipError_t launch_pointwise(const void* x, const void* w, const void* bias, void* y,
                            const Geom& g, hipStream_t s);

bool can_igemm(const Geom& g, int dtype);
hipError_t launch_igemm(const void* x, const void* w, const void* bias, void* y,
                        const Geom& g, hipStream_t s);

bool can_igemm_band(const Geom& g, int dtype);
// Output rows per band (0 when the band kernel declines); automatic
// selection prefers the band kernel from 5 rows on.
bool igemm_band_preferred(const Geom& g);
hipError_t launch_igemm_band(const void* x, const void* w, const void* bias, void* y,
                             const Geom& g, hipStream_t s);

bool can_depthwise(const Geom& g, int dtype);
// Small groups (C/G = C_out/G = 4 or 8, 3x3, bf16, C a multiple of 64) on the
// 4x4x4 matrix instruction; the depthwise path takes it where it applies.
bool can_grouped_mfma(const Geom& g, int dtype);
hipError_t launch_grouped_mfma(const void* x, const void* w, const void* bias, void* y, const Geom& g,
                               hipStream_t s);
hipError_t launch_depthwise(const void* x, const void* w, const void* bias, void* y,
                            const Geom& g, int dtype, hipStream_t s);

// Weight gradient, split over the pixels of the batch into `pieces` pieces of
// `per` pixels whose fp32 partials (pieces x weight elements) go to a
// workspace of `workspace` bytes, then reduced in piece order.
struct DwPlan {
    int64_t per;
    int pieces;
    size_t workspace;
};
DwPlan plan_dw_direct(const Geom& g);
bool can_dw_igemm(const Geom& g, int dtype);
DwPlan plan_dw_igemm(const Geom& g, int cus);
hipError_t launch_dw_igemm(const void* x, const void* dy, void* dw, void* workspace, const Geom& g,
                           int cus, hipStream_t s);
hipError_t launch_dw_direct(const void* x, const void* dy, void* dw, void* workspace,
                            const Geom& g, int dtype, hipStream_t s);
hipError_t launch_dw_reduce(const float* part, void* dw, int64_t wn, int pieces, int dtype,
                            hipStream_t s);

// The fixed device scratch of conv_bwd_dw_noalloc: kScratchBytes bytes,
// 256-byte aligned, one array per device; *out receives this device's
// address (looked up once per device).
constexpr size_t kScratchBytes = size_t(16) << 20;
hipError_t scratch_buffer(void** out);

bool can_dx_igemm(const Geom& g, int dtype);
// Input gradient of small groups (C/G = C_out/G = 1, 2, 4, or 8 in bf16),
// NHWC: per-channel gather on the vector units, per-channel bias.
bool can_dx_depthwise(const Geom& g, int dtype);
hipError_t launch_dx_depthwise(const void* dy, const void* w, const void* bias, void* dx, const Geom& g,
                               int dtype, hipStream_t s);
hipError_t launch_dx_igemm(const void* dy, const void* w, const void* bias, void* dx,
                           const Geom& g, hipStream_t s);
// Input gradient of stride-2, dilation-1 3x3 and 4x4 kernels: all four
// stride phases of a band of rows per workgroup.
bool can_dx_band(const Geom& g, int dtype);
hipError_t launch_dx_band(const void* dy, const void* w, const void* bias, void* dx,
                          const Geom& g, hipStream_t s);

// Sums of fp32 partials in row order, rounded once: column c of `pieces`
// consecutive rows of `pitch` values goes to out[c], for each of `groups`
// groups (of `pieces` rows and `cols` outputs each, one after another).  No
// pieces: zeros.  A null out is skipped.
constexpr int kSumJobs = 6;
struct SumJob {
    const float* part;
    int64_t pitch, cols;
    int pieces, groups;
    void* out;
};
struct SumArgs {
    SumJob job[kSumJobs];
    uint32_t begin[kSumJobs];  // first workgroup (filled at the launch)
    int jobs;
};
inline void add_sum(SumArgs& a, const float* part, int64_t pitch, int64_t cols, int pieces, void* out, int groups = 1)
{
    a.job[a.jobs++] = SumJob{part, pitch, cols, pieces, groups, out};
}
hipError_t launch_sums(SumArgs a, int dtype, hipStream_t s);

// Norms before and after a block with gate and residual scale (see
// conv_block_norm_fwd / conv_block_norm_bwd in include/convmi.h).
struct RowStats {
    float f_mean, f_r, y_mean, y_r, c1, c2;       // what the column sums of a long row need of it
};
struct NormArgs {
    const void *dy, *da;                          // backward only
    const void *x, *f, *z, *s;                    // stream, branch, gate, scale
    const void *post_w, *post_b, *pre_w, *pre_b;
    void *y, *a;                                  // forward
    void *dx, *df, *dz, *ds, *dpost_w, *dpost_b, *dpre_w, *dpre_b;
    float* part;                                  // fp32 partial sums
    RowStats* stats;                              // of long rows, behind them
    int64_t rows, gate_rows;                      // gate_rows: rows that share one gate row
    int C;
    int post, pre, act;
    float eps;
};
hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s);
size_t norm_bwd_workspace(int64_t rows, int C);

// Gated feed-forward layer (see conv_gated_fwd / conv_gated_bwd).
struct GatedArgs {
    const void *dh, *x, *wg, *wu, *bg, *bu;
    float* saved;
    void *h, *dx, *dwg, *dwu, *dbg, *dbu;
    void* workspace;
    int64_t rows;
    int C, F, act;
};
hipError_t launch_gated_fwd(const GatedArgs& a, int dtype, hipStream_t s);
hipError_t launch_gated_bwd(const GatedArgs& a, int dtype, hipStream_t s);
size_t gated_fwd_workspace(int64_t rows, int C, int F, int dtype);
size_t gated_bwd_workspace(int64_t rows, int C, int F, int dtype);

// Global norm of a list of gradients and clipping by it.
constexpr int kClipMaxBlocks = 2048;   // partials of one list of up to kClipTensors tensors
constexpr int kClipTensors = 128;      // tensors one launch takes (its table is a kernel argument)
size_t clip_workspace(int n);
// `dst` null: the norm only.
hipError_t launch_clip(const void* const* src, void* const* dst, const size_t* counts, const int* dtypes, int n,
                       float max_norm, float eps, float* norm, void* workspace, hipStream_t s);

// Short causal convolution along a sequence (see conv_causal_fwd /
// conv_causal_bwd / conv_causal_step).
constexpr int kCausalTaps = 8;         // taps at most
struct CausalArgs {
    const void *x, *w, *bias, *initial, *dy, *dlast;
    const int *starts, *slots;
    void *y, *last, *state, *dx, *dinitial;
    float *part_w, *part_b;            // gradient: partial sums
    int64_t rows, len, xs;             // len: rows of each sequence, without starts; xs: elements from one row of x to the next
    int per;                           // rows of a range
    int seqs, C, K, act, clear;
};
size_t causal_bwd_workspace(int64_t rows, int C, int K);
hipError_t launch_causal_fwd(CausalArgs a, int dtype, hipStream_t s);
hipError_t launch_causal_bwd(CausalArgs a, void* dw, void* db, int dtype, void* workspace, hipStream_t s);
hipError_t launch_causal_step(const CausalArgs& a, int count, int dtype, hipStream_t s);

// Selective state space scan (see conv_scan_fwd / conv_scan_bwd / conv_scan_step).
constexpr int kScanTile = 16;          // rows between two states kept for the gradient
constexpr int kScanStates = 64;        // states of a channel at most
struct ScanArgs {
    const void *x, *delta, *B, *C, *z, *dy;
    const float *A, *D, *bias, *initial, *dlast;
    const int *starts, *slots;
    void *y, *dx, *ddelta, *dB, *dC, *dz;
    float *last, *saved, *dinitial;
    // workspace
    float *ends, *sums;                // a piece's state at its end (or its gradient's at its begin), and sum of d
    float *part_bc, *part_a, *part_d, *part_bias;
    int64_t rows, len;                 // len: rows of each sequence, without starts
    int64_t xs, ds, zs, bs, cs;        // elements from one row to the next
    int64_t piece_rows;
    int64_t part_rows;                 // rows of part_bc
    int64_t sum_rows, row0;            // rows that a launch of the sums of dB and dC adds up, and the first of them
    int seqs, channels, n, groups, per_group;
    int blocks;                        // workgroups of a group's channels
    int pieces;                        // 0: whole sequences, `walk` of them a workgroup
    int walk, seq0;                    // seq0: the first sequence of a launch
    int launch_seqs;                   // sequences of a launch of the gradient
    int softplus, act, clear;          // clear: rows of no sequence become zeros
};
struct ScanGrads {
    float *dA, *dD, *dbias;
};
size_t scan_saved(int64_t rows, int channels, int n);
// `packed`: the sequences' rows are known to the device alone.
size_t scan_fwd_workspace(const ScanArgs& a, bool packed);
size_t scan_bwd_workspace(const ScanArgs& a, bool packed, bool saved);
hipError_t launch_scan_fwd(ScanArgs a, int dtype, void* workspace, hipStream_t s);
hipError_t launch_scan_bwd(ScanArgs a, const ScanGrads& g, int dtype, void* workspace, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, float* state, int count, int dtype, hipStream_t s);

// AdamW over a list of tensors (see conv_adamw).
struct AdamList {
    void *const *params, *const *m, *const *v, *const *copies;
    const void* const* grads;
    float *const *m_scales, *const *v_scales;
    const size_t* counts;
    const int *param_dtypes, *grad_dtypes, *copy_dtypes;
    int n, bits;
};
struct AdamRates {
    double lr, beta1, beta2, eps, weight_decay, max_norm, norm_eps;
    long long step;
    const float *lr_dev, *norm;
    const long long* step_dev;
};
constexpr int kAdamBlock = 128;        // elements that share a scale of 8-bit states
hipError_t launch_adamw(const AdamList& l, const AdamRates& r, hipStream_t s);
hipError_t launch_adamw_moments(const AdamList& l, float* const* m_out, float* const* v_out, hipStream_t s);

}  // namespace convmi
