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
// workgroup sums the same partials, in the same order; and it goes through the
// list backwards, so that what the first pass read last comes out of the
// memory-side cache.  290 tensors, 300M elements, 831 MB: 547 us forwards, 528
// backwards, 495 backwards with streaming stores (5.0 TB/s over the three
// passes).
#include "kernels.hpp"

#include <algorithm>

namespace convmi {
namespace {

constexpr int kThreads = 256;
constexpr size_t kStreamBytes = size_t(128) << 20;

// Up to N tensors.
template <int N>
struct Table {
    const void* src[N];
    void* dst[N];
    uint64_t count[N];        // elements * 2 + (1: bf16, 0: fp32)
    uint32_t begin[N + 1];    // first chunk of each tensor
    int n;
    uint32_t chunk;           // elements in a chunk
};
static_assert(sizeof(Table<kClipTensors>) + 64 <= 4096, "the table is a kernel argument");

// The tensor that holds chunk c.
template <int N>
__device__ __forceinline__ int find(const Table<N>& t, uint32_t c)
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

template <int N>
__global__ __launch_bounds__(kThreads) void clip_norm_kernel(Table<N> t, double* __restrict__ part)
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

template <bool STREAM>
__device__ __forceinline__ void put16(void* p, uint4 v)
{
    uint32x4_any t;
    t.x = v.x; t.y = v.y; t.z = v.z; t.w = v.w;
    if constexpr (STREAM) __builtin_nontemporal_store(t, static_cast<uint32x4_any*>(p));
    else *static_cast<uint32x4_any*>(p) = t;
}

template <bool BF16, bool STREAM>
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
        for (int u = 0; u < U; ++u) put16<STREAM>(q + static_cast<size_t>(i + u * V * kThreads) * E, scaled(v[u], c, BF16));
    }
    for (; i + V <= n; i += V * kThreads)
        store16_any(q + static_cast<size_t>(i) * E, scaled(load16_any(p + static_cast<size_t>(i) * E), c, BF16));
    if (i < n)
        for (; i < n; ++i) {
            if (BF16) store_f(reinterpret_cast<bf16_t*>(q) + i, load_f(reinterpret_cast<const bf16_t*>(p) + i) * c);
            else store_f(reinterpret_cast<float*>(q) + i, load_f(reinterpret_cast<const float*>(p) + i) * c);
        }
}

template <int N, bool STREAM>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(Table<N> t, const double* __restrict__ part, int parts,
                                                              float max_norm, float eps, float* norm)
{
    __shared__ double waves[kThreads / 64];
    const float v = list_norm(part, parts, waves);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float c = max_norm / (v + eps);
    c = c > 1.0f ? 1.0f : c;  // NaN stays
    for (uint32_t i = blockIdx.x; i < t.begin[t.n]; i += gridDim.x) {
        const uint32_t b = t.begin[t.n] - 1 - i;  // from the end
        const int k = find(t, b);
        const char* p = static_cast<const char*>(t.src[k]);
        char* q = static_cast<char*>(t.dst[k]);
        if (c == 1.0f && p == q) continue;  // in place and unclipped: the values stand
        const uint64_t count = t.count[k] >> 1, at = static_cast<uint64_t>(b - t.begin[k]) * t.chunk;
        const uint32_t n = static_cast<uint32_t>(count - at < t.chunk ? count - at : t.chunk);
        if (t.count[k] & 1) chunk_scale<true, STREAM>(p + at * 2, q + at * 2, n, c);
        else chunk_scale<false, STREAM>(p + at * 4, q + at * 4, n, c);
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

namespace {

// One list, N tensors a launch.
template <int N>
hipError_t clip(const void* const* src, void* const* dst, const size_t* counts, const int* dtypes, int n, float max_norm,
                float eps, float* norm, double* part, hipStream_t s)
{
    const int limit = max_blocks(n);
    size_t total = 0, bytes = 0;
    for (int i = 0; i < n; ++i) {
        total += counts[i];
        bytes += counts[i] * (dtypes[i] == 1 ? 2 : 4);
    }
    // A list larger than half of the memory-side cache is written past it, so
    // that the writes leave what the backward walk is about to read.
    auto scale = bytes > kStreamBytes ? clip_scale_kernel<N, true> : clip_scale_kernel<N, false>;
    // Elements in a chunk: about one chunk a workgroup for small lists (from
    // 2048 elements, two vectors a lane in bf16), at most 32768.
    uint32_t chunk = 2048;
    while (chunk < 32768 && total / chunk > static_cast<size_t>(limit)) chunk *= 2;
    Table<N> t;
    auto fill = [&](int i) {  // the tensors from the i-th on; returns the next one
        t.n = 0;
        t.chunk = chunk;
        uint64_t chunks = 0;
        for (; i < n && t.n < N; ++i) {
            if (counts[i] == 0) continue;
            t.src[t.n] = src[i];
            t.dst[t.n] = dst ? dst[i] : nullptr;
            t.count[t.n] = static_cast<uint64_t>(counts[i]) * 2 + (dtypes[i] == 1);
            t.begin[t.n++] = static_cast<uint32_t>(chunks);
            chunks += (counts[i] + chunk - 1) / chunk;
        }
        t.begin[t.n] = static_cast<uint32_t>(chunks);
        return i;
    };
    auto grid = [&] { return dim3(static_cast<unsigned>(std::max<uint32_t>(1, std::min<uint32_t>(t.begin[t.n], limit)))); };
    const ArmedEvents armed = armed_events();
    armed_events() = ArmedEvents{armed.start, nullptr};
    hipError_t e = hipSuccess;
    int parts = 0, i = 0, launches = 0;
    do {
        ++launches;
        i = fill(i);
        const dim3 g = grid();
        e = launch(clip_norm_kernel<N>, g, dim3(kThreads), 0, s, t, part + parts);
        parts += static_cast<int>(g.x);
    } while (e == hipSuccess && i < n);
    armed_events() = ArmedEvents{nullptr, nullptr};
    if (e != hipSuccess) return e;
    if (!dst) {
        armed_events() = ArmedEvents{nullptr, armed.stop};
        e = launch(clip_finish_kernel, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
        armed_events() = ArmedEvents{nullptr, nullptr};
        return e;
    }
    for (int l = launches; e == hipSuccess && l-- > 0;) {
        if (launches > 1) {  // a single launch's table is still there
            i = 0;
            for (int before = 0; before <= l; ++before) i = fill(i);
        }
        if (l == 0) armed_events() = ArmedEvents{nullptr, armed.stop};
        e = launch(scale, grid(), dim3(kThreads), 0, s, t, part, parts, max_norm, eps, l == 0 ? norm : nullptr);
    }
    armed_events() = ArmedEvents{nullptr, nullptr};
    return e;
}

}  // namespace

hipError_t launch_clip(const void* const* src, void* const* dst, const size_t* counts, const int* dtypes, int n,
                       float max_norm, float eps, float* norm, void* workspace, hipStream_t s)
{
    double* part = static_cast<double*>(workspace);
    return n <= 16 ? clip<16>(src, dst, counts, dtypes, n, max_norm, eps, norm, part, s)
                   : clip<kClipTensors>(src, dst, counts, dtypes, n, max_norm, eps, norm, part, s);
}

}  // namespace convmi
