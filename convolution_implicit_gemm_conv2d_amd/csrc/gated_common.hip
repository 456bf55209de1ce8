// The parts of the gated feed-forward layer's gradient that are streams over
// memory, for either type, and the choice between the types.
#include "gated.hpp"

#include <algorithm>

namespace convmi {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load4(const float* p, int n, float* v)
{
    if (n >= 4) {
        const uint4 t = load16_any(p);
        v[0] = __uint_as_float(t.x); v[1] = __uint_as_float(t.y); v[2] = __uint_as_float(t.z); v[3] = __uint_as_float(t.w);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < n ? p[e] : 0.f;
    }
}
__device__ __forceinline__ void load4(const bf16_t* p, int n, float* v)
{
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    if (n >= 4) {
        const u2 t = *reinterpret_cast<const u2*>(p);
        v[0] = __uint_as_float(t.x << 16); v[1] = __uint_as_float(t.x & 0xffff0000u);
        v[2] = __uint_as_float(t.y << 16); v[3] = __uint_as_float(t.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < n ? bf16_to_f(p[e]) : 0.f;
    }
}
__device__ __forceinline__ void put4(float* p, const float* v) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void put4(bf16_t* p, const float* v)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// dg = dh u act'(g), du = dh act(g) from kept g and u.  A stream: 8 bytes
// read and 2 (or 4) read and 4 (or 8) written for an element.  A lane takes
// four hidden channels, a workgroup 256 of them over a chunk of rows, so the
// column sums stay in its registers until the chunk's end.
template <typename T>
__global__ __launch_bounds__(kThreads) void gated_kept_kernel(const T* __restrict__ dh, const float* __restrict__ saved,
                                                              T* __restrict__ d, float* __restrict__ sums, int64_t rows,
                                                              int64_t chunk, int F, int Fp, int act)
{
    __shared__ float4 joined[4][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int f = (blockIdx.x * 64 + lane) * 4;
    const int n = F - f;
    const int64_t r0 = blockIdx.y * chunk, r1 = min(rows, r0 + chunk);
    float sg[4] = {}, su[4] = {};
    with_act(act, [&](auto kind) __attribute__((always_inline)) {
    if (f < Fp) {
#pragma unroll 2
        for (int64_t r = r0 + wave; r < r1; r += 4) {
            float h[4], g[4], u[4], dg[4], du[4];
            load4(dh + r * F + f, n, h);
            load4(saved + r * 2 * F + f, n, g);
            load4(saved + r * 2 * F + F + f, n, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const ActPair p = act_pair<kind()>(g[e]);
                dg[e] = e < n ? h[e] * u[e] * p.d : 0.f;
                du[e] = e < n ? h[e] * p.v : 0.f;
                sg[e] += dg[e];
                su[e] += du[e];
            }
            put4(d + r * 2 * Fp + f, dg);
            put4(d + r * 2 * Fp + Fp + f, du);
        }
    }
    });
    if (!sums) return;
    joined[wave][0][lane] = make_float4(sg[0], sg[1], sg[2], sg[3]);
    joined[wave][1][lane] = make_float4(su[0], su[1], su[2], su[3]);
    __syncthreads();
    if (wave < 2 && f < Fp) {
        float4 t = joined[0][wave][lane];
        for (int w = 1; w < 4; ++w) {
            const float4 o = joined[w][wave][lane];
            t.x += o.x; t.y += o.y; t.z += o.z; t.w += o.w;
        }
        *reinterpret_cast<float4*>(sums + (static_cast<int64_t>(blockIdx.y) * 2 + wave) * Fp + f) = t;
    }
}

}  // namespace

int gated_kept_chunks(int64_t rows, int Fp, int64_t* chunk)
{
    // about eight workgroups a CU, no chunk under 32 rows
    const int64_t cols = (Fp + 255) / 256;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(2048 / cols, rows / 32));
    *chunk = std::max<int64_t>(1, (rows + want - 1) / want);
    return static_cast<int>((rows + *chunk - 1) / *chunk);
}

hipError_t launch_gated_kept(const GatedArgs& a, void* d, float* sums, int Fp, int chunks, int64_t chunk, int dtype,
                             hipStream_t s)
{
    const dim3 grid((Fp + 255) / 256, chunks);
    return dtype ? launch(gated_kept_kernel<bf16_t>, grid, dim3(kThreads), 0, s, static_cast<const bf16_t*>(a.dh), a.saved,
                          static_cast<bf16_t*>(d), sums, a.rows, chunk, a.F, Fp, a.act)
                 : launch(gated_kept_kernel<float>, grid, dim3(kThreads), 0, s, static_cast<const float*>(a.dh), a.saved,
                          static_cast<float*>(d), sums, a.rows, chunk, a.F, Fp, a.act);
}

hipError_t launch_gated_fwd(const GatedArgs& a, int dtype, hipStream_t s)
{
    return dtype ? gated_fwd_bf16(a, s) : gated_fwd_f32(a, s);
}

hipError_t launch_gated_bwd(const GatedArgs& a, int dtype, hipStream_t s)
{
    return dtype ? gated_bwd_bf16(a, s) : gated_bwd_f32(a, s);
}

size_t gated_fwd_workspace(int64_t rows, int C, int F, int dtype)
{
    return dtype ? gated_fwd_workspace_bf16(rows, C, F) : gated_fwd_workspace_f32(rows, C, F);
}

size_t gated_bwd_workspace(int64_t rows, int C, int F, int dtype)
{
    return (dtype ? gated_plan_bf16(rows, C, F) : gated_plan_f32(rows, C, F)).total();
}

}  // namespace convmi
