// Sums of fp32 partial rows in a fixed order, rounded once: the last step of
// gradients whose sums were cut into pieces.  All sums of a call go in one
// launch (a launch costs a small call more than its sums).
//
// A stream over the partials.  Many rows (column sums of rows, cut over the
// device): a workgroup takes 64 columns, its sixteen waves every sixteenth row,
// and the waves' sums are added in order.  Few rows of many columns (partial
// matrices): a lane takes four columns and all rows.  512 rows of 3 x 4096
// columns: 13 us; 16 rows of 2 x 262144 and 784 of 2 x 1024: 8 us.
#include "kernels.hpp"

namespace convmi {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kManyRows = 32;

bool many(const SumJob& j) { return j.pieces >= kManyRows; }

template <typename T>
__global__ __launch_bounds__(kThreads) void sums_kernel(SumArgs a)
{
    __shared__ float sums[kWaves][64];
    int n = 0;
    while (n + 1 < a.jobs && blockIdx.x >= a.begin[n + 1]) ++n;
    const SumJob j = a.job[n];
    const uint32_t block = blockIdx.x - a.begin[n];
    if (j.pieces >= kManyRows) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const uint32_t per = static_cast<uint32_t>((j.cols + 63) / 64), group = block / per;
        const int64_t c = static_cast<int64_t>(block - group * per) * 64 + lane;
        const float* p = j.part + static_cast<int64_t>(group) * j.pieces * j.pitch + c;
        float acc = 0.f;
        if (c < j.cols) {
            constexpr int kBatch = 16;
            for (int s = wave; s < j.pieces; s += kWaves * kBatch) {
                float v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) v[i] = s + kWaves * i < j.pieces ? p[static_cast<int64_t>(s + kWaves * i) * j.pitch] : 0.f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) acc += v[i];
            }
        }
        sums[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && c < j.cols) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) t += sums[w][lane];
            store_f(static_cast<T*>(j.out) + static_cast<int64_t>(group) * j.cols + c, t);
        }
        return;
    }
    const uint32_t per = static_cast<uint32_t>((j.cols + 4 * kThreads - 1) / (4 * kThreads)), group = block / per;
    const int64_t c = (static_cast<int64_t>(block - group * per) * kThreads + threadIdx.x) * 4;
    if (c >= j.cols) return;
    const float* p = j.part + static_cast<int64_t>(group) * j.pieces * j.pitch + c;
    T* out = static_cast<T*>(j.out) + static_cast<int64_t>(group) * j.cols + c;
    const int have = static_cast<int>(j.cols - c < 4 ? j.cols - c : 4);
    if (have == 4) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int kBatch = 8;
        for (int s = 0; s < j.pieces; s += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                v[i] = make_uint4(0, 0, 0, 0);
                if (s + i < j.pieces) v[i] = load16_any(p + static_cast<int64_t>(s + i) * j.pitch);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                acc[0] += __uint_as_float(v[i].x);
                acc[1] += __uint_as_float(v[i].y);
                acc[2] += __uint_as_float(v[i].z);
                acc[3] += __uint_as_float(v[i].w);
            }
        }
        if constexpr (sizeof(T) == 4) {
            store16_any(out, make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])));
        } else {
            typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
            u2 t;
            t.x = pack_bf16x2(acc[0], acc[1]);
            t.y = pack_bf16x2(acc[2], acc[3]);
            *reinterpret_cast<u2*>(out) = t;
        }
    } else {
        for (int e = 0; e < have; ++e) {
            float acc = 0.f;
            for (int s = 0; s < j.pieces; ++s) acc += p[static_cast<int64_t>(s) * j.pitch + e];
            store_f(out + e, acc);
        }
    }
}

}  // namespace

hipError_t launch_sums(SumArgs a, int dtype, hipStream_t s)
{
    int64_t blocks = 0;
    int n = 0;
    for (int i = 0; i < a.jobs; ++i) {
        const SumJob j = a.job[i];
        if (!j.out || j.cols == 0 || j.groups == 0) continue;
        a.job[n] = j;
        a.begin[n++] = static_cast<uint32_t>(blocks);
        const int64_t wide = many(j) ? 64 : 4 * kThreads;
        blocks += (j.cols + wide - 1) / wide * j.groups;
    }
    a.jobs = n;
    if (blocks == 0) return hipSuccess;
    if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    return launch(dtype ? sums_kernel<bf16_t> : sums_kernel<float>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, a);
}

}  // namespace convmi
