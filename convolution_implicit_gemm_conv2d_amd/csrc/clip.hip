// Global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2),
//   c = min(1, max_norm / (norm + eps)),   out = c g.
//
// A NaN or infinite gradient gives a NaN or infinite norm, and c follows the
// formula (infinite: 0, so finite gradients become 0 and infinite ones NaN;
// NaN: everything NaN), so a caller sees it in the norm.
//
// Design.  Both passes are streams over memory (one read; one read and one
// write), so a list costs its bytes plus launches: one launch takes the table
// of up to 128 tensors as its argument, cuts every tensor into chunks of one
// size and gives chunk c to workgroup c mod grid, which finds its tensor by a
// binary search that all lanes share.  Squares are summed in 64 bits: the
// vector units hold that at the memory's rate, a square of a large or tiny
// fp32 gradient neither overflows nor vanishes, and the order of the sums
// (lane, wave, workgroup, list) is fixed, so the norm is the same on every
// run.  The second pass has no launch between it and the first: every
// workgroup sums the same partials, in the same order.
#include "kernels.hpp"

#include <algorithm>

namespace convmi {
namespace {

constexpr int kThreads = 256;

struct Table {
    const void* src[kClipTensors];
    void* dst[kClipTensors];
    uint64_t count[kClipTensors];        // elements * 2 + (1: bf16, 0: fp32)
    uint32_t begin[kClipTensors + 1];    // first chunk of each tensor
    int n;
    uint32_t chunk;                      // elements in a chunk
};
static_assert(sizeof(Table) + 64 <= 4096, "the table is a kernel argument");

// The tensor that holds chunk c.
__device__ __forceinline__ int find(const Table& t, uint32_t c)
{
    int lo = 0, hi = t.n;  // begin[lo] <= c < begin[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.begin[mid] <= c) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v, double* waves)
{
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (waves[0] + waves[1]) + (waves[2] + waves[3]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ double square(float v) { return static_cast<double>(v) * static_cast<double>(v); }

__device__ __forceinline__ double squares(uint4 v, bool bf16, double acc)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            acc += square(__uint_as_float(w[i] << 16));
            acc += square(__uint_as_float(w[i] & 0xffff0000u));
        } else {
            acc += square(__uint_as_float(w[i]));
        }
    }
    return acc;
}

template <bool BF16>
__device__ __forceinline__ double chunk_squares(const char* p, uint32_t n)
{
    constexpr uint32_t V = BF16 ? 8 : 4, E = 16 / V;
    constexpr int U = 4;  // vectors in flight for a lane
    double acc[2] = {0.0, 0.0};
    uint32_t i = threadIdx.x * V;
    for (; i + V * (U * kThreads - kThreads + 1) <= n; i += V * U * kThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load16_any(p + static_cast<size_t>(i + u * V * kThreads) * E);
#pragma unroll
        for (int u = 0; u < U; ++u) acc[u & 1] = squares(v[u], BF16, acc[u & 1]);
    }
    for (; i + V <= n; i += V * kThreads) acc[0] = squares(load16_any(p + static_cast<size_t>(i) * E), BF16, acc[0]);
    if (i < n)  // the tensor's last elements, fewer than a vector
        for (; i < n; ++i)
            acc[1] += square(BF16 ? load_f(reinterpret_cast<const bf16_t*>(p) + i) : load_f(reinterpret_cast<const float*>(p) + i));
    return acc[0] + acc[1];
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(Table t, double* __restrict__ part)
{
    __shared__ double waves[kThreads / 64];
    double acc = 0.0;
    for (uint32_t c = blockIdx.x; c < t.begin[t.n]; c += gridDim.x) {
        const int k = find(t, c);
        const uint64_t count = t.count[k] >> 1, at = static_cast<uint64_t>(c - t.begin[k]) * t.chunk;
        const uint32_t n = static_cast<uint32_t>(count - at < t.chunk ? count - at : t.chunk);
        const char* p = static_cast<const char*>(t.src[k]);
        if (t.count[k] & 1) acc += chunk_squares<true>(p + at * 2, n);
        else acc += chunk_squares<false>(p + at * 4, n);
    }
    acc = block_sum(acc, waves);
    if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm, from all partials of the list; the same in every workgroup.
__device__ __forceinline__ float list_norm(const double* part, int n, double* waves)
{
    double acc = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) acc += part[i];
    return static_cast<float>(sqrt(block_sum(acc, waves)));
}

__global__ __launch_bounds__(kThreads) void clip_finish_kernel(const double* __restrict__ part, int n, float* norm)
{
    __shared__ double waves[kThreads / 64];
    const float v = list_norm(part, n, waves);
    if (threadIdx.x == 0) *norm = v;
}

__device__ __forceinline__ uint4 scaled(uint4 v, float c, bool bf16)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = bf16 ? pack_bf16x2(__uint_as_float(w[i] << 16) * c, __uint_as_float(w[i] & 0xffff0000u) * c)
                    : __float_as_uint(__uint_as_float(w[i]) * c);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ void chunk_scale(const char* p, char* q, uint32_t n, float c)
{
    constexpr uint32_t V = BF16 ? 8 : 4, E = 16 / V;
    constexpr int U = 4;
    uint32_t i = threadIdx.x * V;
    for (; i + V * (U * kThreads - kThreads + 1) <= n; i += V * U * kThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load16_any(p + static_cast<size_t>(i + u * V * kThreads) * E);
#pragma unroll
        for (int u = 0; u < U; ++u) store16_any(q + static_cast<size_t>(i + u * V * kThreads) * E, scaled(v[u], c, BF16));
    }
    for (; i + V <= n; i += V * kThreads)
        store16_any(q + static_cast<size_t>(i) * E, scaled(load16_any(p + static_cast<size_t>(i) * E), c, BF16));
    if (i < n)
        for (; i < n; ++i) {
            if (BF16) store_f(reinterpret_cast<bf16_t*>(q) + i, load_f(reinterpret_cast<const bf16_t*>(p) + i) * c);
            else store_f(reinterpret_cast<float*>(q) + i, load_f(reinterpret_cast<const float*>(p) + i) * c);
        }
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(Table t, const double* __restrict__ part, int parts,
                                                              float max_norm, float eps, float* norm)
{
    __shared__ double waves[kThreads / 64];
    const float v = list_norm(part, parts, waves);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float c = max_norm / (v + eps);
    c = c > 1.0f ? 1.0f : c;  // NaN stays
    for (uint32_t b = blockIdx.x; b < t.begin[t.n]; b += gridDim.x) {
        const int k = find(t, b);
        const char* p = static_cast<const char*>(t.src[k]);
        char* q = static_cast<char*>(t.dst[k]);
        if (c == 1.0f && p == q) continue;  // in place and unclipped: the values stand
        const uint64_t count = t.count[k] >> 1, at = static_cast<uint64_t>(b - t.begin[k]) * t.chunk;
        const uint32_t n = static_cast<uint32_t>(count - at < t.chunk ? count - at : t.chunk);
        if (t.count[k] & 1) chunk_scale<true>(p + at * 2, q + at * 2, n, c);
        else chunk_scale<false>(p + at * 4, q + at * 4, n, c);
    }
}

// Workgroups of a launch: partials of one launch are at most this many.
int max_blocks(int n)
{
    const int launches = std::max(1, (n + kClipTensors - 1) / kClipTensors);
    return std::max(256, kClipMaxBlocks / launches);
}

}  // namespace

size_t clip_workspace(int n)
{
    const int launches = std::max(1, (n + kClipTensors - 1) / kClipTensors);
    return static_cast<size_t>(launches) * max_blocks(n) * sizeof(double);
}

hipError_t launch_clip(const void* const* src, void* const* dst, const size_t* counts, const int* dtypes, int n,
                       float max_norm, float eps, float* norm, void* workspace, hipStream_t s)
{
    double* part = static_cast<double*>(workspace);
    const int limit = max_blocks(n);
    size_t total = 0;
    for (int i = 0; i < n; ++i) total += counts[i];
    // Elements in a chunk: about one chunk a workgroup for small lists (from
    // 2048 elements, two vectors a lane in bf16), at most 32768.
    uint32_t chunk = 2048;
    while (chunk < 32768 && total / chunk > static_cast<size_t>(limit)) chunk *= 2;
    const ArmedEvents armed = armed_events();
    armed_events() = ArmedEvents{armed.start, nullptr};
    int parts = 0;
    for (int pass = 0; pass < (dst ? 2 : 1); ++pass) {
        int at = 0;
        for (int i = 0; i < n || i == 0;) {
            Table t;
            t.n = 0;
            t.chunk = chunk;
            uint64_t chunks = 0;
            for (; i < n && t.n < kClipTensors; ++i) {
                if (counts[i] == 0) continue;
                const uint64_t more = (counts[i] + chunk - 1) / chunk;
                t.src[t.n] = src[i];
                t.dst[t.n] = dst ? dst[i] : nullptr;
                t.count[t.n] = static_cast<uint64_t>(counts[i]) * 2 + (dtypes[i] == 1);
                t.begin[t.n++] = static_cast<uint32_t>(chunks);
                chunks += more;
            }
            t.begin[t.n] = static_cast<uint32_t>(chunks);
            const int grid = static_cast<int>(std::max<uint64_t>(1, std::min<uint64_t>(chunks, limit)));
            const bool last = i >= n;
            hipError_t e;
            if (pass == 0) {
                e = launch(clip_norm_kernel, dim3(grid), dim3(kThreads), 0, s, t, part + at);
                at += grid;
            } else {
                if (last) armed_events() = ArmedEvents{nullptr, armed.stop};
                e = launch(clip_scale_kernel, dim3(grid), dim3(kThreads), 0, s, t, part, parts, max_norm, eps,
                           last ? norm : nullptr);
            }
            if (e != hipSuccess) {
                armed_events() = ArmedEvents{nullptr, nullptr};
                return e;
            }
            if (i >= n) break;
        }
        if (pass == 0) parts = at;
    }
    if (dst) return hipSuccess;
    armed_events() = ArmedEvents{nullptr, armed.stop};
    return launch(clip_finish_kernel, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
}

}  // namespace convmi
