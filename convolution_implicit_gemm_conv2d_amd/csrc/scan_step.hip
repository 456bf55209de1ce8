// Selective scan, a row each of many sequences: the form that answers token by
// token.  Each row's state lies in a slot of a pool and is updated in place.
//
// Bound by the states' stream (read and written once).  A lane holds four states
// of a channel, so a wave reads whole lines; the sum of y goes over the 1 to 16
// lanes of a channel.  Rows that share a slot are taken one after another, by
// the workgroup of the first of them.
#include "act.hpp"
#include "kernels.hpp"
#include "rows_of_slot.hpp"
#include "scan.hpp"

namespace convmi {
namespace scan {
namespace {

constexpr int kPer = 4;  // states of a lane

template <typename T>
__device__ __forceinline__ void step_row(const ScanArgs& a, float* state, int64_t row, int64_t slot, int c, int n0, int lanes)
{
    const bool on = c < a.channels;
    const int cc = on ? c : 0, group = cc / a.per_group;
    float* hp = state + (slot * a.channels + cc) * a.n + n0;
    const float* ap = a.A + static_cast<int64_t>(cc) * a.n + n0;
    const T* bp = static_cast<const T*>(a.B) + row * a.bs + static_cast<int64_t>(group) * a.n + n0;
    const T* cp = static_cast<const T*>(a.C) + row * a.cs + static_cast<int64_t>(group) * a.n + n0;
    const float x = load_f(static_cast<const T*>(a.x) + row * a.xs + cc);
    float d = load_f(static_cast<const T*>(a.delta) + row * a.ds + cc) + (a.bias ? a.bias[cc] : 0.f);
    if (a.softplus) d = softplus<false>(d).v;
    float acc = 0.f;
    auto one = [&](float& h, float A, float b, float cv) __attribute__((always_inline)) {
        h = __builtin_fmaf(exp2_hw(d * (A * kLog2e)), h, d * x * b);
        acc = __builtin_fmaf(h, cv, acc);
    };
    if (on && n0 + kPer <= a.n) {
        const uint4 hv = load16_any(hp), av = load16_any(ap);
        float h[kPer] = {__uint_as_float(hv.x), __uint_as_float(hv.y), __uint_as_float(hv.z), __uint_as_float(hv.w)};
        const float A[kPer] = {__uint_as_float(av.x), __uint_as_float(av.y), __uint_as_float(av.z), __uint_as_float(av.w)};
#pragma unroll
        for (int j = 0; j < kPer; ++j) one(h[j], A[j], load_f(bp + j), load_f(cp + j));
        store16_any(hp, make_uint4(__float_as_uint(h[0]), __float_as_uint(h[1]), __float_as_uint(h[2]), __float_as_uint(h[3])));
    } else if (on) {
        for (int j = 0; j < kPer && n0 + j < a.n; ++j) one(hp[j], ap[j], load_f(bp + j), load_f(cp + j));
    }
    for (int s = 1; s < lanes; s <<= 1) acc += __shfl_xor(acc, s);
    if (on && n0 == 0) {
        float y = a.D ? __builtin_fmaf(a.D[cc], x, acc) : acc;
        if (a.z) y *= act_value(a.act, load_f(static_cast<const T*>(a.z) + row * a.zs + cc));
        store_f(static_cast<T*>(a.y) + row * a.channels + cc, y);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void step_kernel(ScanArgs a, float* state, int count, int lanes, int blocks)
{
    const int row = static_cast<int>(blockIdx.x / blocks);
    const int at = static_cast<int>(blockIdx.x % blocks) * 256 + threadIdx.x;
    const int c = at / lanes, n0 = (at & (lanes - 1)) * kPer;
    each_row_of_slot(a.slots, static_cast<int>(a.rows), count, row, [&](int r, int slot) {
        if (slot >= 0) step_row<T>(a, state, r, slot, c, n0, lanes);
        else if (a.clear && n0 == 0 && c < a.channels) store_f(static_cast<T*>(a.y) + static_cast<int64_t>(r) * a.channels + c, 0.f);
    });
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_step(const ScanArgs& a, float* state, int count, int dtype, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    int lanes = 1;
    while (lanes * scan::kPer < a.n) lanes *= 2;
    const int64_t blocks = (static_cast<int64_t>(a.channels) * lanes + 255) / 256;
    if (blocks * a.rows >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    return launch(dtype ? scan::step_kernel<bf16_t> : scan::step_kernel<float>, dim3(static_cast<unsigned>(blocks * a.rows)), dim3(256), 0, s, a,
                  state, count, lanes, static_cast<int>(blocks));
}

}  // namespace convmi
