// Norms before and after a block, fused with the block's gate, residual scale
// and residual sum; forward and gradient.  For a row of C channels, with f
// the block's output and x the residual stream:
//
//   n = post(f),  y = x + s * act(z) * n,  a = pre(y),
//   rms(v) = v r w, r = 1/sqrt(mean(v^2) + eps);
//   layer(v) = (v - mean(v)) r w + b, r = 1/sqrt(mean((v - mean(v))^2) + eps).
//
// Gradient, from dy and da, with yh and fh the normalised rows, q = da w_pre:
//   D = dy + r_y (q - mean(q) [layer] - yh mean(q yh)),   dx = D,
//   P = D n,  dz = s act'(z) P,  ds = sum act(z) P,  dn = D s act(z),
//   p = dn w_post,  df = r_f (p - mean(p) [layer] - fh mean(p fh)),
//   dw_post = sum dn fh,  db_post = sum dn,  dw_pre = sum da yh,  db_pre = sum da,
// sums over rows; a gate row shared by gate_rows rows sums its dz over them.
//
// What bounds it: memory.  Forward reads x, f (and z) and writes y and a once;
// the gradient reads dy, da, x, f (z) and writes dx, df (dz) once, and works
// the statistics out again, so nothing is kept from the forward pass.  A row
// stays in registers between its reductions (its mean first, then the sum of
// squared differences, both in fp32), a lane holds 8 consecutive channels of
// each of its vectors; rows of up to 1024 channels take one wave, longer ones
// a workgroup.  Rows of odd length load and store the same vectors at
// unaligned addresses; only a row's last, partial vector goes by elements.
//
// Sums over rows: a workgroup walks a contiguous piece of the rows and keeps
// its column sums in registers; pieces write fp32 partials, and a second
// kernel adds them in order.  No atomics, so results do not change from run
// to run.  A piece never holds a part of two shared gate rows unless it holds
// them whole: it either covers whole groups (and writes their dz itself) or a
// part of one (and the second kernel adds the group's parts).
#include "act.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace convmi {
namespace {

constexpr int kVec = 8;  // channels in a lane's vector
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
// Column sums of the gradient, in the order of their blocks in a partial row.
enum { kSumPreW = 0, kSumPostW, kSumScale, kSumPreB, kSumPostB, kSumGate, kSums };

__device__ __forceinline__ void load8(const float* p, int n, float* v)
{
    if (n == kVec) {
        const uint4 a = load16_any(p), b = load16_any(p + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = e < n ? p[e] : 0.f;
    }
}
__device__ __forceinline__ void load8(const bf16_t* p, int n, float* v)
{
    if (n == kVec) {
        const uint4 a = load16_any(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = e < n ? bf16_to_f(p[e]) : 0.f;
    }
}
__device__ __forceinline__ void store8(float* p, int n, const float* v)
{
    if (n == kVec) {
        store16_any(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        store16_any(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) p[e] = v[e];
    }
}
__device__ __forceinline__ void store8(bf16_t* p, int n, const float* v)
{
    if (n == kVec) {
        store16_any(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) p[e] = f_to_bf16(v[e]);
    }
}

// Sum over the lanes that share a row: one wave, or the whole workgroup.
// `slots` alternates between two arrays, so one barrier a sum is enough.
struct RowSum {
    float (*slots)[2][8];  // [2 values][parity][wave]
    int parity;
    template <bool ONE>
    __device__ __forceinline__ float one(float v)
    {
        v = wave_sum(v);
        if (ONE) return v;
        if ((threadIdx.x & 63) == 0) slots[0][parity][threadIdx.x >> 6] = v;
        __syncthreads();
        float t = 0.f;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) t += slots[0][parity][w];
        parity ^= 1;
        return t;
    }
    template <bool ONE>
    __device__ __forceinline__ void two(float& u, float& v)
    {
        u = wave_sum(u);
        v = wave_sum(v);
        if (ONE) return;
        if ((threadIdx.x & 63) == 0) {
            slots[0][parity][threadIdx.x >> 6] = u;
            slots[1][parity][threadIdx.x >> 6] = v;
        }
        __syncthreads();
        u = v = 0.f;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) {
            u += slots[0][parity][w];
            v += slots[1][parity][w];
        }
        parity ^= 1;
    }
};

// A lane's part of a row: VPT vectors of 8 channels, vector i at channel
// (i * lanes + lane) * 8; cnt[i] of its channels exist.
template <int VPT>
struct Part {
    int at[VPT], cnt[VPT];
    __device__ __forceinline__ Part(int C, int lanes, int lane)
    {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            at[i] = (i * lanes + lane) * kVec;
            cnt[i] = min(max(C - at[i], 0), kVec);
        }
    }
};

template <int VPT, typename T>
__device__ __forceinline__ void load_row(const T* p, const Part<VPT>& part, float (&v)[VPT][kVec])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (part.cnt[i] > 0) load8(p + part.at[i], part.cnt[i], v[i]);
        else
            for (int e = 0; e < kVec; ++e) v[i][e] = 0.f;
}
template <int VPT, typename T>
__device__ __forceinline__ void load_param(const T* p, const Part<VPT>& part, float other, float (&v)[VPT][kVec])
{
    if (p) load_row(p, part, v);
    else
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] = e < part.cnt[i] ? other : 0.f;
}
template <int VPT, typename T>
__device__ __forceinline__ void store_row(T* p, const Part<VPT>& part, const float (&v)[VPT][kVec])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (part.cnt[i] > 0) store8(p + part.at[i], part.cnt[i], v[i]);
}

// v *= act(z).
template <int VPT>
__device__ __forceinline__ void times_act(int act, const float (&z)[VPT][kVec], float (&v)[VPT][kVec])
{
    with_act(act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] *= act_value<kind()>(z[i][e]);
    });
}

// Normalises a row in place and returns r; channels past the row stay 0.
template <bool ONE, int VPT>
__device__ __forceinline__ float normalise(int kind, const Part<VPT>& part, float inv_c, float eps, RowSum& rs,
                                           float (&v)[VPT][kVec])
{
    if (kind == kNormLayer) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) t += v[i][e];
        const float mean = rs.one<ONE>(t) * inv_c;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] = e < part.cnt[i] ? v[i][e] - mean : 0.f;
    }
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) t += v[i][e] * v[i][e];
    const float r = 1.0f / sqrtf(rs.one<ONE>(t) * inv_c + eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[i][e] *= r;
    return r;
}

template <typename T, int VPT, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 512) void norm_fwd_kernel(NormArgs k)
{
    __shared__ float slots[2][2][8];
    RowSum rs{slots, 0};
    const int lanes = ONE ? 64 : blockDim.x, lane = ONE ? threadIdx.x & 63 : threadIdx.x;
    const Part<VPT> part(k.C, lanes, lane);
    const float inv_c = 1.0f / k.C;
    const T *x = static_cast<const T*>(k.x), *f = static_cast<const T*>(k.f), *z = static_cast<const T*>(k.z);
    T *y = static_cast<T*>(k.y), *a = static_cast<T*>(k.a);
    const int64_t step = ONE ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
    for (int64_t r = ONE ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x; r < k.rows; r += step) {
        float v[VPT][kVec];
        load_row(x + r * k.C, part, v);
        if (f) {
            float n[VPT][kVec], w[VPT][kVec];
            load_row(f + r * k.C, part, n);
            if (k.post != kNormNone) {
                normalise<ONE>(k.post, part, inv_c, k.eps, rs, n);
                float b[VPT][kVec];
                load_param(static_cast<const T*>(k.post_w), part, 1.f, w);
                load_param(static_cast<const T*>(k.post_b), part, 0.f, b);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) n[i][e] = n[i][e] * w[i][e] + b[i][e];
            }
            if (z) {
                load_row(z + r / k.gate_rows * k.C, part, w);
                times_act(k.act, w, n);
            }
            load_param(static_cast<const T*>(k.s), part, 1.f, w);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[i][e] = e < part.cnt[i] ? v[i][e] + w[i][e] * n[i][e] : 0.f;
        }
        if (y) store_row(y + r * k.C, part, v);
        if (a) {
            float w[VPT][kVec], b[VPT][kVec];
            normalise<ONE>(k.pre, part, inv_c, k.eps, rs, v);
            load_param(static_cast<const T*>(k.pre_w), part, 1.f, w);
            load_param(static_cast<const T*>(k.pre_b), part, 0.f, b);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[i][e] = v[i][e] * w[i][e] + b[i][e];
            store_row(a + r * k.C, part, v);
        }
    }
}

// The pieces of the rows that the gradient's workgroups take.  A shared gate
// row's group is cut into `split` pieces, or (split 1) a piece is `groups`
// whole groups; without a shared gate the rows are one group.
struct Pieces {
    int64_t group;     // rows of a group
    int64_t per;       // rows of a piece
    int64_t groups;    // groups of a piece when it is whole ones
    int split;         // pieces of a group
    int count;
};
Pieces make_pieces(int64_t rows, int64_t gate_rows, int C, bool has_gate)
{
    Pieces p{};
    const bool shared = has_gate && gate_rows > 1;
    p.group = shared ? gate_rows : std::max<int64_t>(rows, 1);
    const int64_t groups = rows / p.group;
    // About four workgroups a CU; fewer where a piece would have too few rows
    // to pay for its partial sums.
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(1024, rows / 8));
    (void)C;
    if (groups <= want) {
        p.groups = 1;
        const int64_t split = std::min<int64_t>(std::max<int64_t>(1, want / std::max<int64_t>(groups, 1)), p.group);
        p.per = (p.group + split - 1) / split;
        p.split = static_cast<int>((p.group + p.per - 1) / p.per);
        p.count = static_cast<int>(groups * p.split);
    } else {
        p.split = 1;
        p.groups = (groups + want - 1) / want;
        p.per = p.groups * p.group;
        p.count = static_cast<int>((groups + p.groups - 1) / p.groups);
    }
    if (rows == 0) p.count = 0;
    return p;
}

// FULL: with bias gradients or a shared gate (three more column sums).
template <typename T, int VPT, bool ONE, bool FULL>
__global__ __launch_bounds__(ONE ? 256 : 512) void norm_bwd_kernel(NormArgs k, Pieces pc)
{
    __shared__ float slots[2][2][8];
    __shared__ float joined[ONE ? 4 : 1][64 * VPT * kVec];
    RowSum rs{slots, 0};
    const int lanes = ONE ? 64 : blockDim.x, lane = ONE ? threadIdx.x & 63 : threadIdx.x;
    const int wave = ONE ? threadIdx.x >> 6 : 0;
    const Part<VPT> part(k.C, lanes, lane);
    const float inv_c = 1.0f / k.C;
    const T *x = static_cast<const T*>(k.x), *f = static_cast<const T*>(k.f), *z = static_cast<const T*>(k.z);
    const T *dy = static_cast<const T*>(k.dy), *da = static_cast<const T*>(k.da);
    T *dx = static_cast<T*>(k.dx), *df = static_cast<T*>(k.df), *dz = static_cast<T*>(k.dz);
    const bool shared = FULL && z && k.gate_rows > 1;
    constexpr int NS = FULL ? kSums : 3;
    float* mine = k.part + static_cast<int64_t>(blockIdx.x) * kSums * k.C;

    float sum[NS][VPT][kVec];
#pragma unroll
    for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum[q][i][e] = 0.f;

    // Adds a column sum over the workgroup's waves (in wave order) and lets
    // `put` have it, in the lanes of wave 0.
    auto join = [&](float (&v)[VPT][kVec], auto put) __attribute__((always_inline)) {
        if constexpr (ONE) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) joined[wave][(i * kVec + e) * 64 + lane] = v[i][e];
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int at = (i * kVec + e) * 64 + lane;
                        v[i][e] = ((joined[0][at] + joined[1][at]) + joined[2][at]) + joined[3][at];
                    }
                put(v);
            }
        } else {
            put(v);
        }
    };

    const int64_t group0 = pc.split > 1 ? blockIdx.x / pc.split : blockIdx.x * pc.groups;
    int64_t r0 = group0 * pc.group + (pc.split > 1 ? (blockIdx.x % pc.split) * pc.per : 0);
    const int64_t end = min(pc.split > 1 ? (group0 + 1) * pc.group : k.rows, r0 + pc.per);
    while (r0 < end) {
        const int64_t stop = shared ? min(end, (r0 / pc.group + 1) * pc.group) : end;
        for (int64_t r = r0 + wave; r < stop; r += ONE ? 4 : 1) {
            float v[VPT][kVec], n[VPT][kVec], g[VPT][kVec], d[VPT][kVec], w[VPT][kVec];
            float rf = 1.f, ry = 1.f;
            // y again: v, with fh in n and s act(z) in g
            load_row(x + r * k.C, part, v);
            if (f) {
                load_row(f + r * k.C, part, n);
                if (k.post != kNormNone) rf = normalise<ONE>(k.post, part, inv_c, k.eps, rs, n);
                load_param(static_cast<const T*>(k.s), part, 1.f, g);
                if (z) {
                    load_row(z + r / k.gate_rows * k.C, part, w);
                    times_act(k.act, w, g);
                }
                float b[VPT][kVec];
                load_param(static_cast<const T*>(k.post_w), part, 1.f, w);
                load_param(static_cast<const T*>(k.post_b), part, 0.f, b);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        v[i][e] = e < part.cnt[i] ? v[i][e] + g[i][e] * (n[i][e] * w[i][e] + b[i][e]) : 0.f;
            }
            // D in d
            load_param(dy ? dy + r * k.C : nullptr, part, 0.f, d);
            if (da) {
                float t[VPT][kVec];
                ry = normalise<ONE>(k.pre, part, inv_c, k.eps, rs, v);
                load_row(da + r * k.C, part, t);
                load_param(static_cast<const T*>(k.pre_w), part, 1.f, w);
                float c1 = 0.f, c2 = 0.f;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        sum[kSumPreW][i][e] += t[i][e] * v[i][e];
                        if (FULL) sum[FULL ? kSumPreB : 0][i][e] += t[i][e];
                        t[i][e] *= w[i][e];
                        c1 += t[i][e];
                        c2 += t[i][e] * v[i][e];
                    }
                rs.two<ONE>(c1, c2);
                c1 = k.pre == kNormLayer ? c1 * inv_c : 0.f;
                c2 *= inv_c;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) d[i][e] += ry * (t[i][e] - c1 - v[i][e] * c2);
            }
            if (dx) store_row(dx + r * k.C, part, d);
            if (!f) continue;
            // gate, scale and branch: fh in n, s act(z) in g, D in d; v is free
            {
                float b[VPT][kVec];
                load_param(static_cast<const T*>(k.post_w), part, 1.f, w);
                load_param(static_cast<const T*>(k.post_b), part, 0.f, b);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[i][e] = d[i][e] * (n[i][e] * w[i][e] + b[i][e]);  // P
            }
            if (z) {
                float t[VPT][kVec], s[VPT][kVec];
                load_row(z + r / k.gate_rows * k.C, part, t);
                load_param(static_cast<const T*>(k.s), part, 1.f, s);
                with_act(k.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const ActPair p = act_pair<kind()>(t[i][e]);
                        if (shared) sum[FULL ? kSumGate : 0][i][e] += v[i][e] * s[i][e] * p.d;
                        else t[i][e] = v[i][e] * s[i][e] * p.d;
                        sum[kSumScale][i][e] += v[i][e] * p.v;
                    }
                });
                if (!shared && dz) store_row(dz + r * k.C, part, t);
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) sum[kSumScale][i][e] += v[i][e];
            }
            float e1 = 0.f, e2 = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float dn = d[i][e] * g[i][e];
                    sum[kSumPostW][i][e] += dn * n[i][e];
                    if (FULL) sum[FULL ? kSumPostB : 0][i][e] += dn;
                    v[i][e] = k.post == kNormNone ? dn : dn * w[i][e];
                    e1 += v[i][e];
                    e2 += v[i][e] * n[i][e];
                }
            if (k.post != kNormNone) {
                rs.two<ONE>(e1, e2);
                e1 = k.post == kNormLayer ? e1 * inv_c : 0.f;
                e2 *= inv_c;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[i][e] = rf * (v[i][e] - e1 - n[i][e] * e2);
            }
            if (df) store_row(df + r * k.C, part, v);
        }
        if (shared) {
            // the group is whole here (split 1): its gate row's gradient is done
            const int64_t group = r0 / pc.group;
            join(sum[FULL ? kSumGate : 0], [&](float (&v)[VPT][kVec]) {
                if (pc.split == 1) {
                    if (dz) store_row(dz + group * k.C, part, v);
                } else {
                    store_row(mine + kSumGate * k.C, part, v);
                }
            });
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) sum[FULL ? kSumGate : 0][i][e] = 0.f;
        }
        r0 = stop;
    }
#pragma unroll
    for (int q = 0; q < (FULL ? kSumGate : 3); ++q)
        join(sum[q], [&](float (&v)[VPT][kVec]) { store_row(mine + q * k.C, part, v); });
}

// Rows too long for the registers: a workgroup walks a row several times,
// whatever its length; later passes find it in the caches.
constexpr int kLongThreads = 512;
struct LongRow {
    const NormArgs& k;
    float inv_c;
    RowSum rs;
    template <typename F>
    __device__ __forceinline__ float sum(F term)
    {
        float t = 0.f;
        for (int c = threadIdx.x; c < k.C; c += kLongThreads) t += term(c);
        return rs.one<false>(t);
    }
    template <typename F>
    __device__ __forceinline__ void stats(int kind, F value, float& mean, float& r)
    {
        mean = 0.f, r = 1.f;
        if (kind == kNormNone) return;
        if (kind == kNormLayer) mean = sum(value) * inv_c;
        const float m = mean;
        r = 1.0f / sqrtf(sum([&](int c) { const float v = value(c) - m; return v * v; }) * inv_c + k.eps);
    }
};
template <typename T>
__device__ __forceinline__ float param(const void* p, int c, float other)
{
    return p ? load_f(static_cast<const T*>(p) + c) : other;
}

template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_fwd_long_kernel(NormArgs k)
{
    __shared__ float slots[2][2][8];
    LongRow row{k, 1.0f / k.C, RowSum{slots, 0}};
    for (int64_t r = blockIdx.x; r < k.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(k.x) + r * k.C;
        const T* f = k.f ? static_cast<const T*>(k.f) + r * k.C : nullptr;
        const T* z = k.z ? static_cast<const T*>(k.z) + r / k.gate_rows * k.C : nullptr;
        float fm = 0.f, fr = 1.f, ym, yr;
        if (f) row.stats(k.post, [&](int c) { return load_f(f + c); }, fm, fr);
        auto value = [&](int c) {
            if (!f) return load_f(x + c);
            float n = load_f(f + c);
            if (k.post != kNormNone) n = (n - fm) * fr * param<T>(k.post_w, c, 1.f) + param<T>(k.post_b, c, 0.f);
            if (z) n *= act_value(k.act, load_f(z + c));
            return load_f(x + c) + param<T>(k.s, c, 1.f) * n;
        };
        if (k.a) {
            row.stats(k.pre, value, ym, yr);
            for (int c = threadIdx.x; c < k.C; c += kLongThreads) {
                const float v = value(c);
                if (k.y) store_f(static_cast<T*>(k.y) + r * k.C + c, v);
                store_f(static_cast<T*>(k.a) + r * k.C + c, (v - ym) * yr * param<T>(k.pre_w, c, 1.f) + param<T>(k.pre_b, c, 0.f));
            }
        } else {
            for (int c = threadIdx.x; c < k.C; c += kLongThreads) store_f(static_cast<T*>(k.y) + r * k.C + c, value(c));
        }
    }
}

// The same walk for the gradient.  A lane owns its channels, so it adds their
// sums up in the workgroup's partial row in memory.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_bwd_long_kernel(NormArgs k, Pieces pc)
{
    __shared__ float slots[2][2][8];
    LongRow row{k, 1.0f / k.C, RowSum{slots, 0}};
    const bool shared = k.z && k.gate_rows > 1;
    float* mine = k.part + static_cast<int64_t>(blockIdx.x) * kSums * k.C;
    for (int c = threadIdx.x; c < k.C; c += kLongThreads)
#pragma unroll
        for (int q = 0; q < kSums; ++q) mine[static_cast<int64_t>(q) * k.C + c] = 0.f;
    const int64_t group0 = pc.split > 1 ? blockIdx.x / pc.split : blockIdx.x * pc.groups;
    const int64_t r0 = group0 * pc.group + (pc.split > 1 ? (blockIdx.x % pc.split) * pc.per : 0);
    const int64_t end = min(pc.split > 1 ? (group0 + 1) * pc.group : k.rows, r0 + pc.per);
    for (int64_t r = r0; r < end; ++r) {
        const T* x = static_cast<const T*>(k.x) + r * k.C;
        const T* f = k.f ? static_cast<const T*>(k.f) + r * k.C : nullptr;
        const T* z = k.z ? static_cast<const T*>(k.z) + r / k.gate_rows * k.C : nullptr;
        const T* dy = k.dy ? static_cast<const T*>(k.dy) + r * k.C : nullptr;
        const T* da = k.da ? static_cast<const T*>(k.da) + r * k.C : nullptr;
        float fm = 0.f, fr = 1.f, ym = 0.f, yr = 1.f, c1 = 0.f, c2 = 0.f, e1 = 0.f, e2 = 0.f;
        if (f) row.stats(k.post, [&](int c) { return load_f(f + c); }, fm, fr);
        auto fh = [&](int c) { return (load_f(f + c) - fm) * fr; };
        auto branch = [&](int c) { return fh(c) * param<T>(k.post_w, c, 1.f) + param<T>(k.post_b, c, 0.f); };
        auto factor = [&](int c) { return param<T>(k.s, c, 1.f) * (z ? act_value(k.act, load_f(z + c)) : 1.f); };
        auto value = [&](int c) { return f ? load_f(x + c) + factor(c) * branch(c) : load_f(x + c); };
        auto q = [&](int c) { return load_f(da + c) * param<T>(k.pre_w, c, 1.f); };
        if (da) {
            row.stats(k.pre, value, ym, yr);
            if (k.pre == kNormLayer) c1 = row.sum(q) * row.inv_c;
            c2 = row.sum([&](int c) { return q(c) * (value(c) - ym) * yr; }) * row.inv_c;
        }
        auto grad = [&](int c) {
            const float d = dy ? load_f(dy + c) : 0.f;
            return da ? d + yr * (q(c) - c1 - (value(c) - ym) * yr * c2) : d;
        };
        auto p = [&](int c) { return grad(c) * factor(c) * param<T>(k.post_w, c, 1.f); };
        if (f && k.post != kNormNone) {
            if (k.post == kNormLayer) e1 = row.sum(p) * row.inv_c;
            e2 = row.sum([&](int c) { return p(c) * fh(c); }) * row.inv_c;
        }
        for (int c = threadIdx.x; c < k.C; c += kLongThreads) {
            const float d = grad(c);
            auto add = [&](int which, float v) { mine[static_cast<int64_t>(which) * k.C + c] += v; };
            if (da) {
                add(kSumPreW, load_f(da + c) * (value(c) - ym) * yr);
                add(kSumPreB, load_f(da + c));
            }
            if (f) {
                const float P = d * branch(c), s = param<T>(k.s, c, 1.f), dn = d * factor(c);
                if (z) {
                    const ActPair a = act_pair(k.act, load_f(z + c));
                    const float g = P * s * a.d;
                    if (shared) add(kSumGate, g);
                    else if (k.dz) store_f(static_cast<T*>(k.dz) + r * k.C + c, g);
                    add(kSumScale, P * a.v);
                } else {
                    add(kSumScale, P);
                }
                add(kSumPostW, dn * fh(c));
                add(kSumPostB, dn);
                if (k.df) {
                    const float t = k.post == kNormNone ? dn : fr * (dn * param<T>(k.post_w, c, 1.f) - e1 - fh(c) * e2);
                    store_f(static_cast<T*>(k.df) + r * k.C + c, t);
                }
            }
            if (k.dx) store_f(static_cast<T*>(k.dx) + r * k.C + c, d);
            if (shared && pc.split == 1 && (r + 1) % pc.group == 0) {
                float& sum = mine[static_cast<int64_t>(kSumGate) * k.C + c];
                if (k.dz) store_f(static_cast<T*>(k.dz) + r / pc.group * k.C + c, sum);
                sum = 0.f;
            }
        }
    }
}

// Adds partial rows: a workgroup takes 64 columns of one output, its waves
// every fourth piece, and the four sums are added in order.
constexpr int kSumThreads = 256;
template <typename T>
__global__ __launch_bounds__(kSumThreads) void column_sums_kernel(SumArgs a)
{
    __shared__ float sums[kSumThreads / 64][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    T* out = static_cast<T*>(a.out[blockIdx.y]);
    if (!out) return;
    float acc = 0.f;
    if (c < a.cols) {
        constexpr int kBatch = 16;
        const float* p = a.part + static_cast<int64_t>(blockIdx.y) * a.q_pitch + c;
        for (int s = wave; s < a.pieces; s += 4 * kBatch) {
            float v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = p[static_cast<int64_t>(min(s + 4 * i, a.pieces - 1)) * a.pitch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s + 4 * i < a.pieces) acc += v[i];
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && c < a.cols) store_f(out + c, ((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane]);
}

// The gate rows of groups that were cut into `split` pieces each.
template <typename T>
__global__ __launch_bounds__(256) void gate_sums_kernel(const float* __restrict__ part, T* __restrict__ dz, int C, int split)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    const float* p = part + (static_cast<int64_t>(blockIdx.y) * split * kSums + kSumGate) * C + c;
    float acc = 0.f;
    for (int s = 0; s < split; ++s) acc += p[static_cast<int64_t>(s) * kSums * C];
    store_f(dz + static_cast<int64_t>(blockIdx.y) * C + c, acc);
}

// Rows of up to this many channels stay in the registers.
constexpr int kRegisterRow = 8192;

template <typename T>
hipError_t fwd(const NormArgs& a, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    const int64_t cus = device_cu_count();
    if (a.C > kRegisterRow)
        return launch(norm_fwd_long_kernel<T>, dim3(std::min<int64_t>(a.rows, cus * 4)), dim3(kLongThreads), 0, s, a);
    if (a.C <= 1024) {
        const unsigned grid = std::min<int64_t>((a.rows + 3) / 4, cus * 8);
        return launch(a.C <= 512 ? norm_fwd_kernel<T, 1, true> : norm_fwd_kernel<T, 2, true>, dim3(grid), dim3(256), 0, s, a);
    }
    const int threads = (a.C + 1023) / 1024 * 64;
    const unsigned grid = std::min<int64_t>(a.rows, cus * 32 / (threads / 64));
    return launch(norm_fwd_kernel<T, 2, false>, dim3(grid), dim3(threads), 0, s, a);
}

template <typename T>
hipError_t bwd(const NormArgs& a, hipStream_t s)
{
    const Pieces pc = make_pieces(a.rows, a.gate_rows, a.C, a.z != nullptr);
    const bool shared = a.z && a.gate_rows > 1;
    const bool full = shared || a.dpre_b || a.dpost_b;
    const ArmedEvents armed = armed_events();
    armed_events() = ArmedEvents{armed.start, nullptr};
    hipError_t e = hipSuccess;
    if (pc.count > 0) {
        const dim3 grid(pc.count);
        if (a.C > kRegisterRow) {
            e = launch(norm_bwd_long_kernel<T>, grid, dim3(kLongThreads), 0, s, a, pc);
        } else if (a.C <= 1024) {
            if (a.C <= 512)
                e = launch(full ? norm_bwd_kernel<T, 1, true, true> : norm_bwd_kernel<T, 1, true, false>, grid, dim3(256), 0, s, a, pc);
            else
                e = launch(full ? norm_bwd_kernel<T, 2, true, true> : norm_bwd_kernel<T, 2, true, false>, grid, dim3(256), 0, s, a, pc);
        } else {
            const int threads = (a.C + 1023) / 1024 * 64;
            e = launch(full ? norm_bwd_kernel<T, 2, false, true> : norm_bwd_kernel<T, 2, false, false>, grid, dim3(threads), 0, s, a, pc);
        }
    }
    armed_events() = ArmedEvents{nullptr, nullptr};
    if (e != hipSuccess) return e;
    if (shared && a.dz && pc.split > 1) {
        const dim3 grid((a.C + 255) / 256, static_cast<unsigned>(a.rows / pc.group));
        e = launch(gate_sums_kernel<T>, grid, dim3(256), 0, s, a.part, static_cast<T*>(a.dz), a.C, pc.split);
        if (e != hipSuccess) return e;
    }
    SumArgs sums{};
    sums.part = a.part;
    sums.pitch = static_cast<int64_t>(kSums) * a.C;
    sums.q_pitch = a.C;
    sums.pieces = pc.count;
    sums.cols = a.C;
    sums.dtype = sizeof(T) == 2;
    void* out[kSumOutputs] = {a.dpre_w, a.dpost_w, a.ds, a.dpre_b, a.dpost_b, nullptr};
    int nq = 0;
    for (int q = 0; q < kSumOutputs; ++q) {
        sums.out[q] = out[q];
        if (out[q]) nq = q + 1;
    }
    armed_events() = ArmedEvents{nullptr, armed.stop};
    if (nq) e = launch_column_sums(sums, nq, s);
    armed_events() = ArmedEvents{nullptr, nullptr};
    return e;
}

}  // namespace

hipError_t launch_column_sums(const SumArgs& a, int nq, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>((a.cols + 63) / 64), nq);
    return a.dtype ? launch(column_sums_kernel<bf16_t>, grid, dim3(kSumThreads), 0, s, a)
                   : launch(column_sums_kernel<float>, grid, dim3(kSumThreads), 0, s, a);
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s)
{
    return dtype ? fwd<bf16_t>(a, s) : fwd<float>(a, s);
}

size_t norm_bwd_workspace(int64_t rows, int64_t gate_rows, int C, int has_gate)
{
    const Pieces pc = make_pieces(rows, gate_rows, C, has_gate != 0);
    return static_cast<size_t>(pc.count) * kSums * C * sizeof(float);
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s)
{
    return dtype ? bwd<bf16_t>(a, s) : bwd<float>(a, s);
}

}  // namespace convmi
