// Selective scan, a row each of many sequences: the form that answers token by
// token.  Each row's state lies in a slot of a pool and is updated in place.
//
// Bound by the states' stream (read and written once) and, with few rows, by
// latency.  A lane holds four states of a channel, so a wave reads whole lines; the sum
// of y goes over the 1 to 16 lanes of a channel.  Rows that share a slot are taken one after another, by
// the workgroup of the first of them.
#include "act.hpp"
#include "kernels.hpp"
#include "rows_of_slot.hpp"
#include "scan.hpp"

namespace convmi {
namespace scan {
namespace {

constexpr int kPer = 4;  // states of a lane

// Four neighbouring values at any alignment.
__device__ __forceinline__ void load4(const float* p, float* v)
{
    const uint4 t = load16_any(p);
    v[0] = __uint_as_float(t.x); v[1] = __uint_as_float(t.y); v[2] = __uint_as_float(t.z); v[3] = __uint_as_float(t.w);
}
__device__ __forceinline__ void load4(const bf16_t* p, float* v)
{
    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
    const u2_any t = *reinterpret_cast<const u2_any*>(p);
    v[0] = __uint_as_float(t.x << 16); v[1] = __uint_as_float(t.x & 0xffff0000u);
    v[2] = __uint_as_float(t.y << 16); v[3] = __uint_as_float(t.y & 0xffff0000u);
}
// WHOLE: the states are a multiple of four, and `have` is 4 or less than 1.
template <bool WHOLE, typename P>
__device__ __forceinline__ void load_states(const P* p, int have, float* v)
{
    if constexpr (WHOLE) {
        load4(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = load_f(p + (j < have ? j : 0));
    }
}

// A row's inputs and states for U channels of a lane, `apart` channels from one
// to the next, with the states from `first` on.
template <typename T, int U, bool WHOLE>
struct Step {
    float h[U][kPer], A[U][kPer], b[U][kPer], c[U][kPer], x[U], d[U], z[U];

    // Lanes behind the states, and channels behind the last, read what is there.
    __device__ __forceinline__ void read(const ScanArgs& a, const float* state, int64_t row, int64_t slot, int c0, int apart, int first)
    {
        const int have = a.n - first, n0 = have > 0 ? first : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = c0 + u * apart < a.channels ? c0 + u * apart : 0, group = ch / a.per_group;
            const int64_t at = static_cast<int64_t>(ch) * a.n + n0;
            load_states<WHOLE>(state + slot * a.channels * a.n + at, have, h[u]);
            load_states<WHOLE>(a.A + at, have, A[u]);
            load_states<WHOLE>(static_cast<const T*>(a.B) + row * a.bs + static_cast<int64_t>(group) * a.n + n0, have, b[u]);
            load_states<WHOLE>(static_cast<const T*>(a.C) + row * a.cs + static_cast<int64_t>(group) * a.n + n0, have, c[u]);
            x[u] = load_f(static_cast<const T*>(a.x) + row * a.xs + ch);
            d[u] = load_f(static_cast<const T*>(a.delta) + row * a.ds + ch) + (a.bias ? a.bias[ch] : 0.f);
            z[u] = a.z ? load_f(static_cast<const T*>(a.z) + row * a.zs + ch) : 0.f;
        }
    }
    __device__ __forceinline__ void finish(const ScanArgs& a, float* state, int64_t row, int64_t slot, int c0, int apart, int first, int lanes)
    {
        const int have = a.n - first;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = c0 + u * apart;
            const bool on = ch < a.channels;
            const float t = a.softplus ? softplus<false>(d[u]).v : d[u];
            float y = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                h[u][j] = __builtin_fmaf(exp2_hw(t * (A[u][j] * kLog2e)), h[u][j], t * x[u] * b[u][j]);
                if (j < have) y = __builtin_fmaf(h[u][j], c[u][j], y);
            }
            float* to = state + (slot * a.channels + ch) * a.n + first;
            if constexpr (WHOLE) {
                if (on && have > 0)
                    store16_any(to, make_uint4(__float_as_uint(h[u][0]), __float_as_uint(h[u][1]), __float_as_uint(h[u][2]), __float_as_uint(h[u][3])));
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (on && j < have) to[j] = h[u][j];
            }
            for (int s = 1; s < lanes; s <<= 1) y += __shfl_xor(y, s);
            if (on && first == 0) {
                if (a.D) y = __builtin_fmaf(a.D[ch], x[u], y);
                if (a.z) y *= act_value(a.act, z[u]);
                store_f(static_cast<T*>(a.y) + row * a.channels + ch, y);
            }
        }
    }
};

template <typename T, int U, bool WHOLE>
__global__ __launch_bounds__(256) void step_kernel(ScanArgs a, float* state, int count, int lanes, int blocks, int row0)
{
    const int row = row0 + static_cast<int>(blockIdx.x / blocks);
    const int at = static_cast<int>(blockIdx.x % blocks) * (256 * U) + threadIdx.x;
    const int c = at / lanes, apart = 256 / lanes, first = (at & (lanes - 1)) * kPer;
    Step<T, U, WHOLE> step;
    each_row_of_slot(
        a.slots, static_cast<int>(a.rows), count, row, [&](int r, int slot) { step.read(a, state, r, slot, c, apart, first); },
        [&](int r, int slot) { step.finish(a, state, r, slot, c, apart, first, lanes); },
        [&](int r) {
            if (!a.clear || first != 0) return;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * apart < a.channels) store_f(static_cast<T*>(a.y) + static_cast<int64_t>(r) * a.channels + c + u * apart, 0.f);
        });
}

template <typename T>
auto kernel_of(bool two, bool whole)
{
    return whole ? (two ? step_kernel<T, 2, true> : step_kernel<T, 1, true>) : two ? step_kernel<T, 2, false> : step_kernel<T, 1, false>;
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_step(const ScanArgs& a, float* state, int count, int dtype, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    int lanes = 1;
    while (lanes * scan::kPer < a.n) lanes *= 2;
    // Two channels a lane where the workgroups still fill the device (64 rows of
    // 4096 channels, 16 states: 12.6 us with one, 12.0 with two, 15.1 with four).
    const int64_t all = static_cast<int64_t>(a.channels) * lanes, half = (all + 511) / 512;
    const bool two = half * a.rows >= 1024;
    const int64_t blocks = two ? half : (all + 255) / 256;
    auto kernel = dtype ? scan::kernel_of<bf16_t>(two, a.n % scan::kPer == 0) : scan::kernel_of<float>(two, a.n % scan::kPer == 0);
    return in_grids(blocks * a.rows, 256, blocks, [&](int64_t first, dim3 grid) {
        return launch(kernel, grid, dim3(256), 0, s, a, state, count, lanes, static_cast<int>(blocks), static_cast<int>(first / blocks));
    });
}

}  // namespace convmi
