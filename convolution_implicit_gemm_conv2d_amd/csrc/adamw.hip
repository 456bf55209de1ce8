// AdamW over a list of tensors, with states in 32 or in 8 bits.
//
//   c = min(1, max_norm / (norm + norm_eps)),  g' = c g,
//   m' = b1 m + (1 - b1) g',   v' = b2 v + (1 - b2) g'^2,
//   p' = p (1 - lr w) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
//
// A stream over memory: every parameter, gradient and state is read once and
// what changes is written once (fp32 throughout: 28 bytes an element; bf16 with
// 8-bit states: 10).  Clipping by a norm in hand costs a factor here, where
// clip_gradients is a pass of its own.  One launch takes a table of up to 48
// tensors as its argument and has a workgroup for each chunk of them.  250 M elements
// of mixed types: 1075 to 1100 us with 32-bit states (5.9 TB/s); 795 to 825 with 8-bit ones,
// which their roots and borders bound, and 505 to 520 to read those out.
//
// 8 bits: 128 elements, on 32 lanes, share a scale.  m is the scale times q |q|
// and the root of v the scale times q^2: steps next to the largest value are
// 1.6 % and 3.1 % and values down to 6e-5 (of the root of v 1.5e-5) of it still have a code of
// their own, without a table.  A value next to a border is compared with it
// exactly, so codes do not depend on the roundings of the hardware's root and
// reciprocal, and the arithmetic up to them has a fixed order of roundings, no
// multiply-add contracted.
#include "adamw_tables.hpp"
#include "kernels.hpp"

#include <cmath>

namespace convmi {
namespace {

constexpr int kThreads = kAdamThreads, kE = kAdamElements;
constexpr float kTiny = 0x1p-100f;     // blocks below it hold zeros
constexpr int kMostM = 127, kMostV = 255;

constexpr uint32_t kChunk = kAdamChunk;

template <int N>
struct Table {
    void *p[N], *m[N], *v[N], *copy[N];
    const void* g[N];
    float *ms[N], *vs[N];
    uint64_t count[N];        // elements * 8 + (1: p bf16) + (2: g bf16) + (4: copy bf16)
    uint32_t begin[N + 1];    // first chunk of each tensor
    int n;
};
constexpr int kTensors = 48;
static_assert(sizeof(Table<kTensors>) + 128 <= 4096, "the table is a kernel argument");
// Lists that fit a table of a KiB take one: a launch hands its whole argument to the
// device, whatever is in it (a tensor of 1000 elements 5.2 us so and 5.9 with the large
// table, 12 of them 6.5 and 6.9).
constexpr int kFewTensors = 14;
static_assert(sizeof(Table<kFewTensors>) <= 1024 && sizeof(Table<kFewTensors + 1>) > 1024, "as many as a KiB holds");

struct Rates {
    double lr, log_b1, log_b2;         // for device values
    float keep, rate, root, eps;       // 1 - lr w, lr / (1 - b1^t), (1 - b2^t)^-1/2
    float b1, c1, b2, c2, max_norm, norm_eps;
    double weight_decay;
    long long step;
    const float *lr_dev, *norm;
    const long long* step_dev;
};

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

// kE elements from the i-th on; past the `have`-th zeros.
typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
template <bool STREAM, typename W>
__device__ __forceinline__ W get(const W* p)
{
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool STREAM, typename W>
__device__ __forceinline__ void set(W* p, W w)
{
    if constexpr (STREAM) __builtin_nontemporal_store(w, p);
    else *p = w;
}
template <bool STREAM>
__device__ __forceinline__ void load_e(const void* at, bool bf16, uint64_t i, int have, float* v)
{
    if (have >= kE) {
        if (bf16) {
            const u2_any w = get<STREAM>(reinterpret_cast<const u2_any*>(static_cast<const bf16_t*>(at) + i));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        } else {
            const uint32x4_any w = get<STREAM>(reinterpret_cast<const uint32x4_any*>(static_cast<const float*>(at) + i));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(w[k]);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        v[k] = 0.f;
        if (k < have) v[k] = bf16 ? load_f(static_cast<const bf16_t*>(at) + i + k) : load_f(static_cast<const float*>(at) + i + k);
    }
}
template <bool STREAM>
__device__ __forceinline__ void store_e(void* at, bool bf16, uint64_t i, int have, const float* v)
{
    if (have >= kE) {
        if (bf16) {
            u2_any w;
#pragma unroll
            for (int k = 0; k < 2; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
            set<STREAM>(reinterpret_cast<u2_any*>(static_cast<bf16_t*>(at) + i), w);
        } else {
            uint32x4_any w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(v[k]);
            set<STREAM>(reinterpret_cast<uint32x4_any*>(static_cast<float*>(at) + i), w);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kE; ++k)
        if (k < have) {
            if (bf16) store_f(static_cast<bf16_t*>(at) + i + k, v[k]);
            else store_f(static_cast<float*>(at) + i + k, v[k]);
        }
}

typedef uint32_t word_any __attribute__((aligned(1)));
__device__ __forceinline__ uint32_t load_codes(const void* at, uint64_t i, int have)
{
    const uint8_t* p = static_cast<const uint8_t*>(at) + i;
    if (have >= kE) return *reinterpret_cast<const word_any*>(p);
    uint32_t q = 0;
#pragma unroll
    for (int k = 0; k < kE; ++k)
        if (k < have) q |= static_cast<uint32_t>(p[k]) << (8 * k);
    return q;
}
__device__ __forceinline__ void store_codes(void* at, uint64_t i, int have, uint32_t q)
{
    uint8_t* p = static_cast<uint8_t*>(at) + i;
    if (have >= kE) {
        *reinterpret_cast<word_any*>(p) = q;
    } else {
#pragma unroll
        for (int k = 0; k < kE; ++k)
            if (k < have) p[k] = static_cast<uint8_t>(q >> (8 * k));
    }
}

// Over the 32 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
#define CONVMI_MAX(CTRL) v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false)))
    CONVMI_MAX(0x128);
    CONVMI_MAX(0x124);
    CONVMI_MAX(0x122);
    CONVMI_MAX(0x121);
#undef CONVMI_MAX
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // the other row of 16
    return max(static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1]));
}

#pragma clang fp contract(off)

__device__ __forceinline__ float m_of(uint32_t byte, float scale)
{
    const float q = static_cast<float>(static_cast<int8_t>(byte));
    return q * fabsf(q) * scale;
}
__device__ __forceinline__ float v_of(uint32_t byte, float scale)
{
    const float q = static_cast<float>(byte), r = q * q * scale;
    return r * r;
}
__device__ __forceinline__ void decode(uint32_t qm, uint32_t qv, float km, float kv, float* m, float* v)
{
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        m[k] = m_of((qm >> (8 * k)) & 255u, km);
        v[k] = v_of((qv >> (8 * k)) & 255u, kv);
    }
}

// Codes of a block's m and v, and its scales.
__device__ __forceinline__ void encode(const float* m, const float* v, uint32_t& qm, uint32_t& qv, float& km, float& kv)
{
    uint32_t top_m = 0, top_v = 0;  // as bits: a NaN is above everything
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        top_m = max(top_m, __float_as_uint(m[k]) & 0x7fffffffu);
        top_v = max(top_v, __float_as_uint(v[k]) & 0x7fffffffu);
    }
    const float sm = __uint_as_float(block_max(top_m)), sv = __uint_as_float(block_max(top_v));
    km = sm < kTiny ? 0.f : sm * (1.0f / 16129.0f);
    kv = sv < kTiny ? 0.f : __builtin_sqrtf(sv) * (1.0f / 65025.0f);
    // The hardware's root takes denormal values for 0: small blocks' v are lifted.
    const bool small = sv < 0x1p-40f;
    const float lift = small ? 0x1p64f : 1.0f;
    // No scale, or one that is no number: all codes are 0, but for a positive v under an
    // infinite scale, which keeps its 1.  Either way a block whose scale is not finite
    // stands for no finite value: 0 times it is NaN.
    const float im = km > 0.f ? __builtin_amdgcn_rcpf(km) : 0.f, iv = kv > 0.f ? __builtin_amdgcn_rcpf(kv) * (small ? 0x1p-32f : 1.0f) : 0.f;
    const float most_m = km > 0.f && km < __builtin_inff() ? kMostM : 0.f, most_v = kv > 0.f && kv < __builtin_inff() ? kMostV : 0.f;
    qm = qv = 0;
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        // The guess is off by 2e-4 at most (two roundings of the reciprocal and
        // the root each, at codes up to 255), so only values within 1e-3 of a
        // border are compared with it.
        const float a = fabsf(m[k]), t = __builtin_amdgcn_sqrtf(a * im), r = __builtin_rintf(t);
        float c = __builtin_fminf(r, most_m);
        if (fabsf(t - r) > 0.499f) {
            const float up = c + 0.5f, down = c - 0.5f;
            if (a > up * up * km && c < kMostM) c += 1.0f;
            else if (c > 0.f && !(a > down * down * km)) c -= 1.0f;
        }
        const int q = static_cast<int>(c);
        qm |= (static_cast<uint32_t>(m[k] < 0.f ? -q : q) & 255u) << (8 * k);
        const float tv = __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v[k] * lift) * iv), rv = __builtin_rintf(tv);
        float d = __builtin_fminf(rv, most_v);
        if (fabsf(tv - rv) > 0.499f) {
            const float up = (d + 0.5f) * (d + 0.5f) * kv, down = (d - 0.5f) * (d - 0.5f) * kv;
            if (v[k] > up * up && d < kMostV) d += 1.0f;
            else if (d > 0.f && !(v[k] > down * down)) d -= 1.0f;
        }
        const uint32_t w = static_cast<uint32_t>(d);
        qv |= (w == 0 && v[k] > 0.f && kv > 0.f ? 1u : w) << (8 * k);
    }
}

// m', v' and p' of one element; a fixed order of roundings up to m' and v'.
__device__ __forceinline__ void update(float& p, float g, float& m, float& v, float clip, const Rates& r)
{
    g = g * clip;
    m = m * r.b1 + g * r.c1;
    v = v * r.b2 + g * r.c2 * g;
    const bool small = v < 0x1p-64f;  // the hardware's root takes denormal values for 0
    const float d = __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.0f) * r.root + r.eps;
    p = p * r.keep - m * r.rate * __builtin_amdgcn_rcpf(d);
}

template <int BITS, int N, bool STREAM>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table<N> t, Rates r)
{
    __shared__ float late[3];
    if (r.lr_dev || r.step_dev) {
        if (threadIdx.x == 0) {
            const double lr = r.lr_dev ? static_cast<double>(*r.lr_dev) : r.lr;
            const double step = static_cast<double>(r.step_dev ? *r.step_dev : r.step);
            late[0] = static_cast<float>(1.0 - lr * r.weight_decay);
            late[1] = static_cast<float>(lr / (1.0 - exp(step * r.log_b1)));
            late[2] = static_cast<float>(1.0 / sqrt(1.0 - exp(step * r.log_b2)));
        }
        __syncthreads();
        r.keep = late[0];
        r.rate = late[1];
        r.root = late[2];
    }
    float clip = 1.0f;
    if (r.norm) {
        clip = r.max_norm / (*r.norm + r.norm_eps);
        clip = clip > 1.0f ? 1.0f : clip;  // NaN stays
    }
    const int k = find(t, blockIdx.x);
    const uint64_t count = t.count[k] >> 3, first = static_cast<uint64_t>(blockIdx.x - t.begin[k]) * kChunk;
    const uint32_t n = static_cast<uint32_t>(count - first < kChunk ? count - first : kChunk), at = threadIdx.x * kE;
    // With 8 bits all lanes of a block of 128 go through its step together.
    if ((BITS == 8 ? at & ~static_cast<uint32_t>(kAdamBlock - 1) : at) >= n) return;
    const bool pb = t.count[k] & 1, gb = t.count[k] & 2, cb = t.count[k] & 4;
    const int have = at < n ? static_cast<int>(n - at < kE ? n - at : kE) : 0;
    const uint64_t i = first + at;
    float p[kE], g[kE], m[kE], v[kE];
    load_e<STREAM>(t.p[k], pb, i, have, p);
    load_e<STREAM>(t.g[k], gb, i, have, g);
    if constexpr (BITS == 8) {
        decode(load_codes(t.m[k], i, have), load_codes(t.v[k], i, have), t.ms[k][i / kAdamBlock], t.vs[k][i / kAdamBlock], m, v);
    } else {
        load_e<STREAM>(t.m[k], false, i, have, m);
        load_e<STREAM>(t.v[k], false, i, have, v);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) update(p[e], g[e], m[e], v[e], clip, r);
    store_e<STREAM>(t.p[k], pb, i, have, p);
    if (t.copy[k]) store_e<STREAM>(t.copy[k], cb, i, have, p);
    if constexpr (BITS == 8) {
#pragma unroll
        for (int e = 0; e < kE; ++e)
            if (e >= have) m[e] = v[e] = 0.f;
        uint32_t qm, qv;
        float km, kv;
        encode(m, v, qm, qv, km, kv);
        store_codes(t.m[k], i, have, qm);
        store_codes(t.v[k], i, have, qv);
        if ((threadIdx.x & (kAdamBlock / kE - 1)) == 0) {
            t.ms[k][i / kAdamBlock] = km;
            t.vs[k][i / kAdamBlock] = kv;
        }
    } else {
        store_e<STREAM>(t.m[k], false, i, have, m);
        store_e<STREAM>(t.v[k], false, i, have, v);
    }
}

// p: m's values, copy: v's values.
template <int N, bool STREAM>
__global__ __launch_bounds__(kThreads) void moments_kernel(Table<N> t)
{
    const int k = find(t, blockIdx.x);
    const uint64_t count = t.count[k] >> 3, first = static_cast<uint64_t>(blockIdx.x - t.begin[k]) * kChunk;
    const uint32_t n = static_cast<uint32_t>(count - first < kChunk ? count - first : kChunk), at = threadIdx.x * kE;
    if (at >= n) return;
    const int have = static_cast<int>(n - at < kE ? n - at : kE);
    const uint64_t i = first + at;
    float m[kE], v[kE];
    decode(load_codes(t.m[k], i, have), load_codes(t.v[k], i, have), t.ms[k][i / kAdamBlock], t.vs[k][i / kAdamBlock], m, v);
    store_e<STREAM>(t.p[k], false, i, have, m);
    store_e<STREAM>(t.copy[k], false, i, have, v);
}

// Lists whose step moves more than half of the memory-side cache go past it both
// ways: nothing in it would be there at the next step (250 M elements, 32-bit
// states: 1247 us with ordinary accesses, 1251 with streaming stores, 1129 with
// streaming loads too).
constexpr size_t kStreamBytes = size_t(128) << 20;
bool streams(const AdamList& l)
{
    size_t bytes = 0;
    for (int i = 0; i < l.n; ++i) bytes += l.counts[i] * (l.bits == 8 ? 12 : 28);
    return bytes > kStreamBytes;
}

// One list, tables of N tensors: `go` launches one.
template <int N, typename Go>
hipError_t each_table(const AdamList& l, float* const* m_out, float* const* v_out, Go go)
{
    hipError_t e = hipSuccess;
    CallEvents events;
    ListPlace at;
    while (e == hipSuccess && more_chunks(l.counts, l.n, at)) {
        Table<N> t;
        t.n = 0;
        const int sb = l.bits == 8 ? 1 : 4;  // bytes of a state
        auto plus = [](void* p, uint64_t bytes) { return p ? static_cast<void*>(static_cast<char*>(p) + bytes) : nullptr; };
        const uint32_t chunks = fill_table(l.counts, l.n, N, kMostChunks, at, [&](int k, int i, uint64_t first, uint64_t count, uint32_t begin) {
            t.m[k] = plus(l.m[i], first * sb);
            t.v[k] = plus(l.v[i], first * sb);
            t.ms[k] = l.m_scales ? l.m_scales[i] + first / kAdamBlock : nullptr;
            t.vs[k] = l.v_scales ? l.v_scales[i] + first / kAdamBlock : nullptr;
            t.count[k] = count * 8;
            if (m_out) {
                t.p[k] = m_out[i] + first;
                t.copy[k] = v_out[i] + first;
                t.g[k] = nullptr;
            } else {
                const bool pb = l.param_dtypes[i] == 1, gb = l.grad_dtypes[i] == 1, cb = l.copies && l.copies[i] && l.copy_dtypes[i] == 1;
                t.p[k] = plus(l.params[i], first * (pb ? 2 : 4));
                t.g[k] = plus(const_cast<void*>(l.grads[i]), first * (gb ? 2 : 4));
                t.copy[k] = l.copies ? plus(l.copies[i], first * (cb ? 2 : 4)) : nullptr;
                t.count[k] += (pb ? 1 : 0) + (gb ? 2 : 0) + (cb ? 4 : 0);
            }
            t.begin[k] = begin;
            t.n = k + 1;
        });
        t.begin[t.n] = chunks;
        events.next(!more_chunks(l.counts, l.n, at));
        e = go(t, dim3(chunks));
    }
    return e;
}

}  // namespace

hipError_t launch_adamw(const AdamList& l, const AdamRates& a, hipStream_t s)
{
    Rates r{};
    r.lr = a.lr;
    r.weight_decay = a.weight_decay;
    r.step = a.step;
    r.log_b1 = std::log(a.beta1);
    r.log_b2 = std::log(a.beta2);
    const double t = static_cast<double>(a.step);
    r.keep = static_cast<float>(1.0 - a.lr * a.weight_decay);
    r.rate = static_cast<float>(a.lr / (1.0 - std::pow(a.beta1, t)));
    r.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, t)));
    r.eps = static_cast<float>(a.eps);
    r.b1 = static_cast<float>(a.beta1);
    r.c1 = static_cast<float>(1.0 - a.beta1);
    r.b2 = static_cast<float>(a.beta2);
    r.c2 = static_cast<float>(1.0 - a.beta2);
    r.max_norm = static_cast<float>(a.max_norm);
    r.norm_eps = static_cast<float>(a.norm_eps);
    r.lr_dev = a.lr_dev;
    r.step_dev = a.step_dev;
    r.norm = a.norm;
    const bool stream = streams(l);
    auto run = [&](auto small) {
        constexpr int N = decltype(small)::value;
        auto kernel = l.bits == 8 ? (stream ? adamw_kernel<8, N, true> : adamw_kernel<8, N, false>) : stream ? adamw_kernel<32, N, true> : adamw_kernel<32, N, false>;
        return each_table<N>(l, nullptr, nullptr, [&](const Table<N>& t, dim3 grid) { return launch(kernel, grid, dim3(kThreads), 0, s, t, r); });
    };
    return l.n <= kFewTensors ? run(std::integral_constant<int, kFewTensors>{}) : run(std::integral_constant<int, kTensors>{});
}

hipError_t launch_adamw_moments(const AdamList& l, float* const* m_out, float* const* v_out, hipStream_t s)
{
    const bool stream = streams(l);
    auto run = [&](auto small) {
        constexpr int N = decltype(small)::value;
        return each_table<N>(l, m_out, v_out, [&](const Table<N>& t, dim3 grid) { return launch(stream ? moments_kernel<N, true> : moments_kernel<N, false>, grid, dim3(kThreads), 0, s, t); });
    };
    return l.n <= kFewTensors ? run(std::integral_constant<int, kFewTensors>{}) : run(std::integral_constant<int, kTensors>{});
}

}  // namespace convmi
