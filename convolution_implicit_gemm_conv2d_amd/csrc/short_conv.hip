// Short causal convolution of every channel along its sequence, with an
// activation, states before and behind, its gradient, and a form for tokens.
//
//   p[t] = b + sum_k w[k] x[t - K + 1 + k],   y[t] = act(p[t]),
// rows before a sequence's first from its initial state (zeros without one).
// Gradient: dp = dy act'(p) (p again from x), dx[t] = sum_k w[k] dp[t + K - 1 - k]
// over the rows of the sequence, dw[k] = sum_t dp[t] x[t - K + 1 + k], db = sum_t dp[t].
//
// A stream over memory: a lane takes four neighbouring channels and walks down a
// range of rows with the last K - 1 rows (in the gradient also the last K - 1
// dp) in registers, so every value is loaded once but for the K - 1 rows around
// a range.  The next four rows' loads are out while four are worked on (72 -> 58
// us for 4 x 4096 rows of 4096 channels, bf16: 4.7 TB/s; training step of 20011 packed rows of
// 1544 channels: 31 us forward, 64 the gradient at two waves a SIMD, 6 the sums).  Sequences may begin anywhere in a range.  The rows' ragged end
// repeats channels of the lane before it.
#include "act.hpp"
#include "kernels.hpp"
#include "rows_of_slot.hpp"

#include <algorithm>

namespace convmi {
namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;  // rows loaded at once

// V neighbouring values: as loaded, and in fp32.
template <int N>
struct Words {
    typedef uint32_t any __attribute__((ext_vector_type(N), aligned(2)));
};
template <>
struct Words<1> {
    typedef uint32_t any __attribute__((aligned(2)));
};
template <typename T, int V>
struct Vec {
    static constexpr int N = V * static_cast<int>(sizeof(T)) / 4;  // dwords
    uint32_t w[N];
    __device__ __forceinline__ void load(const T* p)
    {
        const typename Words<N>::any t = *reinterpret_cast<const typename Words<N>::any*>(p);
        if constexpr (N == 1) w[0] = t;
        else
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = t[i];
    }
    __device__ __forceinline__ void open(float* v) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ void load(const T* p, float* v)
    {
        Vec t;
        t.load(p);
        t.open(v);
    }
    static __device__ __forceinline__ void store(T* p, const float* v)
    {
        typename Words<N>::any t;
        if constexpr (sizeof(T) == 4) {
            if constexpr (N == 1) t = __float_as_uint(v[0]);
            else
#pragma unroll
                for (int i = 0; i < N; ++i) t[i] = __float_as_uint(v[i]);
        } else if constexpr (N == 1) {
            t = pack_bf16x2(v[0], v[1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
        *reinterpret_cast<typename Words<N>::any*>(p) = t;
    }
};
// A single value of bf16.
template <>
struct Vec<bf16_t, 1> {
    bf16_t w;
    __device__ __forceinline__ void load(const bf16_t* p) { w = *p; }
    __device__ __forceinline__ void open(float* v) const { v[0] = bf16_to_f(w); }
    static __device__ __forceinline__ void load(const bf16_t* p, float* v) { v[0] = load_f(p); }
    static __device__ __forceinline__ void store(bf16_t* p, const float* v) { store_f(p, v[0]); }
};

struct Span {
    int64_t begin, end;
};
__device__ __forceinline__ Span span_of(const CausalArgs& a, int s)
{
    if (!a.starts) return {s * a.len, (s + 1) * a.len};
    // whatever the offsets hold, the rows are the tensor's
    int64_t b = a.starts[s], e = a.starts[s + 1];
    b = b < 0 ? 0 : b > a.rows ? a.rows : b;
    e = e < b ? b : e > a.rows ? a.rows : e;
    return {b, e};
}
// The first sequence that ends behind `row`.
__device__ __forceinline__ int first_of(const CausalArgs& a, int64_t row)
{
    if (!a.starts) return static_cast<int>(row / a.len);
    int lo = 0, hi = a.seqs;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);  // lo + hi may pass 2^31
        if (span_of(a, mid).end > row) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// A lane's channels and their K taps.
template <typename T, int V, int K>
struct Taps {
    int c;
    float w[K][V], b[V];
    __device__ Taps(const CausalArgs& a, int vec)
    {
        c = V == 1 ? vec : (vec * V + V <= a.C ? vec * V : a.C - V);
        const T *wp = static_cast<const T*>(a.w) + static_cast<int64_t>(c) * K, *bp = static_cast<const T*>(a.bias) + c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b[v] = a.bias ? load_f(bp + v) : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                w[k][v] = load_f(wp + v * K + k);
            }
        }
    }
    __device__ const T* x(const CausalArgs& a, int64_t row) const { return static_cast<const T*>(a.x) + row * a.xs + c; }
    // The row at `pos` of a sequence, also before its first one.
    __device__ void before(const CausalArgs& a, int s, const Span& span, int64_t pos, float* v) const
    {
        if (pos >= 0) {
            Vec<T, V>::load(x(a, span.begin + pos), v);
        } else if (a.initial && pos > -K) {
            Vec<T, V>::load(static_cast<const T*>(a.initial) + (static_cast<int64_t>(s) * (K - 1) + (K - 1 + pos)) * a.C + c, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.f;
        }
    }
};

template <typename T, int V>
__device__ __forceinline__ void put_zeros(void* p, int64_t row, int C, int c)
{
    const float zero[V] = {};
    Vec<T, V>::store(static_cast<T*>(p) + row * C + c, zero);
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void causal_fwd_kernel(CausalArgs a, int64_t ranges, int vecs)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, range = at / vecs;
    if (range >= ranges + (a.last ? a.seqs : 0)) return;
    const Taps<T, V, K> t(a, static_cast<int>(at - range * vecs));
    if (range >= ranges) {  // the last rows of a sequence
        const int s = static_cast<int>(range - ranges);
        const Span span = span_of(a, s);
        for (int j = 0; j < K - 1; ++j) {
            float v[V];
            t.before(a, s, span, span.end - span.begin - (K - 1) + j, v);
            Vec<T, V>::store(static_cast<T*>(a.last) + (static_cast<int64_t>(s) * (K - 1) + j) * a.C + t.c, v);
        }
        return;
    }
    const int64_t first = range * a.per, stop = first + a.per < a.rows ? first + a.per : a.rows;
    T* y = static_cast<T*>(a.y);
    int64_t row = first;
    for (int s = first_of(a, first); s < a.seqs && row < stop; ++s) {
        const Span span = span_of(a, s);
        if (a.clear)
            for (; row < span.begin && row < stop; ++row) put_zeros<T, V>(y, row, a.C, t.c);
        row = span.begin > row ? span.begin : row;
        const int64_t end = span.end < stop ? span.end : stop;
        if (row >= end) continue;
        float win[K - 1 + kU][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) t.before(a, s, span, row - span.begin - (K - 1) + k, win[k]);
        // The next rows' loads run beside these rows' work; rows past the end
        // are the last one again.
        Vec<T, V> next[kU];
        auto load = [&](int64_t from) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kU; ++u) next[u].load(t.x(a, from + u < end ? from + u : end - 1));
        };
        load(row);
        for (; row < end; row += kU) {
            const int n = static_cast<int>(end - row < kU ? end - row : kU);
#pragma unroll
            for (int u = 0; u < kU; ++u) next[u].open(win[K - 1 + u]);
            load(row + kU);
            float p[kU][V];
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    p[u][v] = t.b[v];
#pragma unroll
                    for (int k = 0; k < K; ++k) p[u][v] = __builtin_fmaf(t.w[k][v], win[u + k][v], p[u][v]);
                }
            with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int v = 0; v < V; ++v) p[u][v] = act_value<kind()>(p[u][v]);
            });
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (u < n) Vec<T, V>::store(y + (row + u) * a.C + t.c, p[u]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = win[k + kU][v];
        }
        row = end;
    }
    if (a.clear)
        for (; row < stop; ++row) put_zeros<T, V>(y, row, a.C, t.c);
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void causal_bwd_kernel(CausalArgs a, int64_t ranges, int vecs)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, range = at / vecs;
    if (range >= ranges + (a.dinitial ? a.seqs : 0)) return;
    const Taps<T, V, K> t(a, static_cast<int>(at - range * vecs));
    const T* dy = static_cast<const T*>(a.dy);
    const int before = K - 1;

    // Rows of x and dy, on their way; rows from `stop` on are the one before it.
    Vec<T, V> next_x[kU], next_g[kU];
    auto load = [&](int64_t row, int64_t stop) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t r = row + u < stop ? row + u : stop - 1;
            next_x[u].load(t.x(a, r));
            next_g[u].load(dy + r * a.C + t.c);
        }
    };
    // dp of the loaded rows, `n` of which are there: p again from the window,
    // times dy.
    auto take = [&](float (*win)[V], float (*g)[V]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            next_x[u].open(win[before + u]);
            next_g[u].open(g[u]);
        }
    };
    auto slopes = [&](float (*win)[V], float (*g)[V], int n, float (*dp)[V]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dp[u][v] = t.b[v];
#pragma unroll
                for (int k = 0; k < K; ++k) dp[u][v] = __builtin_fmaf(t.w[k][v], win[u + k][v], dp[u][v]);
            }
        with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) dp[u][v] = u < n ? g[u][v] * act_pair<kind()>(dp[u][v]).d : 0.f;
        });
    };
    // The gradient of the last rows that reaches position `pos` of sequence s.
    auto add_last = [&](int s, const Span& span, int64_t pos, float* d) __attribute__((always_inline)) {
        const int64_t j = pos - (span.end - span.begin) + (K - 1);
        if (!a.dlast || j < 0) return;
        float v[V];
        Vec<T, V>::load(static_cast<const T*>(a.dlast) + (static_cast<int64_t>(s) * (K - 1) + j) * a.C + t.c, v);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += v[i];
    };

    if (range >= ranges) {  // a sequence's initial state: its first rows' dp, and the last rows of a short one
        const int s = static_cast<int>(range - ranges);
        const Span span = span_of(a, s);
        const int64_t len = span.end - span.begin;
        float win[K - 1 + kU][V], d[K - 1][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            t.before(a, s, span, k - before, win[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) d[k][v] = 0.f;
        }
#pragma unroll
        for (int row = 0; row < K - 1; row += kU) {
            const int n = static_cast<int>(len - row < 0 ? 0 : len - row < kU ? len - row : kU);
            float dp[kU][V], g[kU][V];
            if (n == 0) break;
            load(span.begin + row, span.begin + row + n);
            take(win, g);
            slopes(win, g, n, dp);
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int k = 0; k < K - 1; ++k)  // row + u reads position k - (K - 1) by its tap k - row - u
                    if (k - row - u >= 0)
#pragma unroll
                        for (int v = 0; v < V; ++v) d[k][v] = __builtin_fmaf(t.w[k - row - u >= 0 ? k - row - u : 0][v], dp[u][v], d[k][v]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = win[k + kU][v];
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            add_last(s, span, k - before, d[k]);
            Vec<T, V>::store(static_cast<T*>(a.dinitial) + (static_cast<int64_t>(s) * (K - 1) + k) * a.C + t.c, d[k]);
        }
        return;
    }
    const int64_t first = range * a.per, stop = first + a.per < a.rows ? first + a.per : a.rows;
    T* dx = static_cast<T*>(a.dx);
    float dw[K][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][v] = 0.f;
    }
    int64_t row = first;
    for (int s = first_of(a, first); s < a.seqs && row < stop; ++s) {
        const Span span = span_of(a, s);
        if (a.clear && dx)
            for (; row < span.begin && row < stop; ++row) put_zeros<T, V>(dx, row, a.C, t.c);
        row = span.begin > row ? span.begin : row;
        const int64_t end = span.end < stop ? span.end : stop, begin = row;
        if (row >= end) continue;
        // K - 1 rows behind the range's last one still read its rows
        const int64_t far = span.end < end + before ? span.end : end + before;
        float win[K - 1 + kU][V], back[K - 1 + kU][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            t.before(a, s, span, row - span.begin - before + k, win[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) back[k][v] = 0.f;
        }
        load(row, far);
        for (; row < end + before; row += kU) {
            const int n = static_cast<int>(far - row < 0 ? 0 : far - row < kU ? far - row : kU);
            const int own = static_cast<int>(end - row < 0 ? 0 : end - row < kU ? end - row : kU);
            float g[kU][V];
            take(win, g);
            load(row + kU, far);
            slopes(win, g, n, back + before);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (u < own)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += back[before + u][v];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][v] = __builtin_fmaf(back[before + u][v], win[u + k][v], dw[k][v]);
                    }
                const int64_t to = row + u - before;  // complete with this row's dp
                if (dx && to >= begin && to < end) {
                    float d[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        d[v] = 0.f;
#pragma unroll
                        for (int k = 0; k < K; ++k) d[v] = __builtin_fmaf(t.w[k][v], back[before + u - k][v], d[v]);
                    }
                    add_last(s, span, to - span.begin, d);
                    Vec<T, V>::store(dx + to * a.C + t.c, d);
                }
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[k][v] = win[k + kU][v];
                    back[k][v] = back[k + kU][v];
                }
        }
        row = end;
    }
    if (a.clear && dx)
        for (; row < stop; ++row) put_zeros<T, V>(dx, row, a.C, t.c);
    float* pw = a.part_w + (range * a.C + t.c) * K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            pw[v * K + k] = dw[k][v];
        }
        a.part_b[range * a.C + t.c + v] = db[v];
    }
}

// A row each of many sequences; the K - 1 rows before it in a slot of a pool.
template <typename T>
__global__ __launch_bounds__(kThreads) void causal_step_kernel(CausalArgs a, int count, int blocks, int row0)
{
    const int row = row0 + static_cast<int>(blockIdx.x / blocks), c = static_cast<int>(blockIdx.x % blocks) * kThreads + threadIdx.x;
    const bool on = c < a.C;
    const int K = a.K, cc = on ? c : 0;  // lanes behind the last channel read the first one
    T x = T(0), old[kCausalTaps - 1], w[kCausalTaps], b = T(0);
    auto at = [&](int slot) { return static_cast<T*>(a.state) + static_cast<int64_t>(slot) * (K - 1) * a.C + cc; };
    each_row_of_slot(
        a.slots, static_cast<int>(a.rows), count, row,
        [&](int r, int slot) {
            const T* state = at(slot);
            x = static_cast<const T*>(a.x)[r * a.xs + cc];
#pragma unroll
            for (int k = 0; k < kCausalTaps - 1; ++k)
                if (k < K - 1) old[k] = state[static_cast<int64_t>(k) * a.C];
#pragma unroll
            for (int k = 0; k < kCausalTaps; ++k)
                if (k < K) w[k] = static_cast<const T*>(a.w)[static_cast<int64_t>(cc) * K + k];
            if (a.bias) b = static_cast<const T*>(a.bias)[cc];
        },
        [&](int r, int slot) {
            if (!on) return;
            T* state = at(slot);
            float p = load_f(&b), last = 0.f;
#pragma unroll
            for (int k = 0; k < kCausalTaps; ++k)
                if (k < K) {
                    if (k < K - 1) p = __builtin_fmaf(load_f(&w[k]), load_f(&old[k < kCausalTaps - 1 ? k : 0]), p);
                    else last = load_f(&w[k]);
                    if (k > 0 && k < K - 1) state[static_cast<int64_t>(k - 1) * a.C] = old[k < kCausalTaps - 1 ? k : 0];
                }
            p = __builtin_fmaf(last, load_f(&x), p);
            state[static_cast<int64_t>(K - 2) * a.C] = x;
            store_f(static_cast<T*>(a.y) + static_cast<int64_t>(r) * a.C + c, act_value(a.act, p));
        },
        [&](int r) {
            if (on && a.clear) store_f(static_cast<T*>(a.y) + static_cast<int64_t>(r) * a.C + c, 0.f);
        });
}

// Channels of a lane: four, or one where there are fewer.  Two would leave room
// for more waves, but are slower both ways (65 us for 58, 118 for 113).
int vector_of(const CausalArgs& a) { return a.C >= 4 ? 4 : 1; }

// Rows of a range: the fewest that leave no more lanes than the device holds at
// four waves a SIMD.  Fewer rows are read twice and have more partial sums, more
// leave SIMDs empty (4 x 4096 rows of 4096 channels: 61, 58 and 62 us with 32, 64
// and 128 rows; training step of 20011 rows of 1544 channels: 130, 113 and 129 us
// with 16, 32 and 64).
void plan(CausalArgs& a)
{
    const int64_t vecs = (a.C + vector_of(a) - 1) / vector_of(a);
    a.per = 8;
    while (a.per < 128 && (a.rows + a.per - 1) / a.per * vecs > 262144) a.per *= 2;
}

size_t up(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

size_t causal_bwd_workspace(int64_t rows, int C, int K)
{
    CausalArgs a{};
    a.rows = rows;
    a.C = C;
    plan(a);
    const size_t ranges = static_cast<size_t>((rows + a.per - 1) / a.per);
    return up(ranges * C * K * 4) + up(ranges * C * 4);
}

#define CONVMI_TAPS(T, V, KERNEL, GO)                 \
    switch (a.K) {                                    \
    case 2: e = GO((KERNEL<T, V, 2>)); break;         \
    case 3: e = GO((KERNEL<T, V, 3>)); break;         \
    case 4: e = GO((KERNEL<T, V, 4>)); break;         \
    case 5: e = GO((KERNEL<T, V, 5>)); break;         \
    case 6: e = GO((KERNEL<T, V, 6>)); break;         \
    case 7: e = GO((KERNEL<T, V, 7>)); break;         \
    default: e = GO((KERNEL<T, V, 8>)); break;        \
    }
#define CONVMI_CAUSAL(KERNEL, GO)                                                                                 \
    if (dtype) {                                                                                                  \
        if (vector_of(a) == 4) { CONVMI_TAPS(bf16_t, 4, KERNEL, GO) } else { CONVMI_TAPS(bf16_t, 1, KERNEL, GO) } \
    } else {                                                                                                      \
        if (vector_of(a) == 4) { CONVMI_TAPS(float, 4, KERNEL, GO) } else { CONVMI_TAPS(float, 1, KERNEL, GO) }   \
    }

// The launches of `ranges` ranges and then `states` sequences' states, `vecs` lanes
// each, as a grid holds them (fewer than 2^32 lanes; the ranges alone have 2^18, or
// rows * channels / 512).  A later launch is given the ranges less what is behind
// it, a negative number, and so goes on at a sequence.
template <typename Go>
hipError_t each_grid(int64_t ranges, int64_t states, int64_t vecs, CallEvents& events, bool last, Go go)
{
    constexpr int64_t kMost = (int64_t(1) << 32) - kThreads;
    if (ranges > kMost / vecs) return hipErrorInvalidConfiguration;
    hipError_t e = hipSuccess;
    for (int64_t lanes; ranges + states > 0 && e == hipSuccess; ranges -= lanes / vecs) {
        const int64_t all = (ranges + states) * vecs;
        lanes = all < kMost ? all : kMost;
        events.next(last && lanes == all);
        e = go(ranges, dim3(static_cast<unsigned>((lanes + kThreads - 1) / kThreads)));
    }
    return e;
}

hipError_t launch_causal_fwd(CausalArgs a, int dtype, hipStream_t s)
{
    plan(a);
    const int64_t ranges = (a.rows + a.per - 1) / a.per, vecs = (a.C + vector_of(a) - 1) / vector_of(a);
    CallEvents events;
    return each_grid(ranges, a.last ? a.seqs : 0, vecs, events, true, [&](int64_t at, dim3 grid) {
        hipError_t e = hipSuccess;
#define GO(k) launch(k, grid, dim3(kThreads), 0, s, a, at, static_cast<int>(vecs))
        CONVMI_CAUSAL(causal_fwd_kernel, GO)
        return e;
    });
}

hipError_t launch_causal_bwd(CausalArgs a, void* dw, void* db, int dtype, void* workspace, hipStream_t s)
{
    plan(a);
    const int64_t ranges = (a.rows + a.per - 1) / a.per, vecs = (a.C + vector_of(a) - 1) / vector_of(a);
    if (ranges >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    a.part_w = static_cast<float*>(workspace);
    a.part_b = reinterpret_cast<float*>(static_cast<char*>(workspace) + up(static_cast<size_t>(ranges) * a.C * a.K * 4));
    SumArgs sums{};
    const int64_t wn = static_cast<int64_t>(a.C) * a.K;
    if (dw) add_sum(sums, a.part_w, wn, wn, static_cast<int>(ranges), dw);
    if (db) add_sum(sums, a.part_b, a.C, a.C, static_cast<int>(ranges), db);
    CallEvents events;
    const hipError_t rc = each_grid(ranges, a.dinitial ? a.seqs : 0, vecs, events, !sums.jobs, [&](int64_t at, dim3 grid) {
        hipError_t e = hipSuccess;
        CONVMI_CAUSAL(causal_bwd_kernel, GO)
        return e;
    });
    if (rc != hipSuccess || !sums.jobs) return rc;
    events.next(true);
    return launch_sums(sums, dtype, s);
}
#undef GO

hipError_t launch_causal_step(const CausalArgs& a, int count, int dtype, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    const int64_t blocks = (a.C + kThreads - 1) / kThreads;
    return in_grids(blocks * a.rows, kThreads, blocks, [&](int64_t first, dim3 grid) {
        return launch(dtype ? causal_step_kernel<bf16_t> : causal_step_kernel<float>, grid, dim3(kThreads), 0, s, a, count, static_cast<int>(blocks),
                      static_cast<int>(first / blocks));
    });
}

}  // namespace convmi
