// Shared by the gated feed-forward layer's bf16 and fp32 kernels: the plan of
// the gradient's workspace and the entry points of either type.
#pragma once

#include "act.hpp"
#include "kernels.hpp"

namespace convmi {

// The gradient's workspace: dg and du as rows [2 * Fp] of the type (Fp: F
// rounded up so that a K tile never holds both), partial column sums of dg and
// du, and fp32 partials of dx and of the weight gradients, where their sums are
// cut into pieces, and copies of x and the weights with padded rows.
struct GatedPlan {
    int Fp;
    int sum_rows;          // partial rows of the column sums, [2][Fp] each
    int pieces;            // of the weight gradients' sum; 1: no partials
    int64_t per;           // rows of a piece
    int tile;              // and the product's tile
    int x_pieces;          // of dx's sum, values of a piece, tile
    int64_t x_per;
    int x_tile;
    size_t d_bytes, sum_bytes, x_bytes, w_bytes, pad_bytes;
    size_t total() const { return d_bytes + sum_bytes + x_bytes + w_bytes + pad_bytes; }
};
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

hipError_t gated_fwd_bf16(const GatedArgs& a, hipStream_t s);
hipError_t gated_bwd_bf16(const GatedArgs& a, hipStream_t s);
GatedPlan gated_plan_bf16(int64_t rows, int C, int F);
size_t gated_fwd_workspace_bf16(int64_t rows, int C, int F);
hipError_t gated_fwd_f32(const GatedArgs& a, hipStream_t s);
hipError_t gated_bwd_f32(const GatedArgs& a, hipStream_t s);
GatedPlan gated_plan_f32(int64_t rows, int C, int F);
size_t gated_fwd_workspace_f32(int64_t rows, int C, int F);

// dg and du from kept projections: d[row] = [dg | du], with partial column
// sums of `chunk` rows each when sums is not null.
hipError_t launch_gated_kept(const GatedArgs& a, void* d, float* sums, int Fp, int chunks, int64_t chunk, int dtype,
                             hipStream_t s);
int gated_kept_chunks(int64_t rows, int Fp, int64_t* chunk);

}  // namespace convmi
