// Norms before and after a block, fused with its gate, residual scale
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
// squared differences, both in fp32).  A lane holds 8 consecutive channels of
// each of its vectors; rows of up to 512 channels share a wave with others (8,
// 16, 32 or 64 lanes each), longer ones take a workgroup.
// Parameters stay in registers or LDS over a workgroup's rows, and a row's loads go
// out before the row before it is worked on.
//
// A row whose length is no multiple of 8 ends in a vector that starts early
// and repeats channels of the one before: whole loads and stores (at any
// alignment, both lanes store the same values) and only the row sums leave the
// repeated channels out.
//
// Sums over rows: a workgroup walks a contiguous piece of the rows and keeps
// its column sums in registers; pieces write fp32 partials, and a second
// kernel adds them in order.  No atomics, so results do not change from run
// to run.  A piece never holds a part of two shared gate rows unless it holds
// them whole: it either covers whole groups (and writes their dz itself) or a
// part of one (and the second kernel adds the group's parts).
#include "act.hpp"
#include "kernels.hpp"
#include "row_walk.hpp"

#include <algorithm>
#include <atomic>
#include <limits>
#include <type_traits>

namespace convmi {
namespace {

constexpr int kVec = 8;  // channels in a lane's vector
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
// Column sums of the gradient, in the order of their blocks in a partial row.
enum { kSumPreW = 0, kSumPostW, kSumScale, kSumPreB, kSumPostB, kSumGate, kSums };

// A tensor's rows from a (uniform) one on: a buffer, so that all tensors of a
// call share a lane's one offset and a lane without channels of its own needs
// no branch (its offset is past the end: loads give zeros, stores are dropped).
constexpr uint32_t kAll = 0x7ffffffcu;
template <typename T>
__device__ __forceinline__ rsrc_t rows_from(const void* p, int64_t at)
{
    return make_rsrc(static_cast<const T*>(p) + at, kAll);
}

// Eight values as they lie in memory.
template <typename T>
struct Raw {
    static constexpr int kWords = sizeof(T) / 2;
    uint4 u[kWords];
    __device__ __forceinline__ void load(rsrc_t r, uint32_t off)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) u[i] = buffer_load16(r, off + i * 16);
    }
    __device__ __forceinline__ void get(float (&v)[kVec]) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint4 a = u[0], b = u[kWords - 1];
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        }
    }
    // Keeps the compiler from unpacking a parameter once for all rows, which
    // takes twice the registers in bf16.
    __device__ __forceinline__ void stay()
    {
        if constexpr (sizeof(T) == 2) asm volatile("" : "+v"(u[0].x), "+v"(u[0].y), "+v"(u[0].z), "+v"(u[0].w));
    }
    __device__ __forceinline__ void fill(float t)
    {
        const uint32_t w = sizeof(T) == 2 ? pack_bf16x2(t, t) : __float_as_uint(t);
#pragma unroll
        for (int i = 0; i < kWords; ++i) u[i] = make_uint4(w, w, w, w);
    }
};
template <typename T>
__device__ __forceinline__ void store8(rsrc_t r, uint32_t off, const float (&v)[kVec])
{
    if constexpr (sizeof(T) == 2) {
        buffer_store16(r, off, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    } else {
        buffer_store16(r, off, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        buffer_store16(r, off + 16, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    }
}

// Sum over groups of L lanes of a wave, the same in every lane of a group.
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    v += dpp_shift<0xb1, 0xf>(v);            // i ^ 1
    v += dpp_shift<0x4e, 0xf>(v);            // i ^ 2
    v += dpp_shift<0x141, 0xf>(v);           // 7 - i
    if (L >= 16) v += dpp_shift<0x140, 0xf>(v);  // 15 - i
    if (L >= 32) {
        const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    }
    if (L >= 64) {
        const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    }
    return v;
}

// Sums over the lanes that share a row: L of them in a wave, or (L 0) the
// workgroup.  `slots` alternates between two arrays, so one barrier a sum is
// enough.
constexpr int kMaxWaves = 16;
template <int L>
struct RowSum {
    float (*slots)[2][kMaxWaves];  // [2 values][parity][wave]
    int parity;
    __device__ __forceinline__ float total(int which) const
    {
        float t = 0.f;
        const int waves = blockDim.x >> 6;
        for (int w = 0; w < waves; w += 4) {  // slots past the last wave hold 0
            const float4 s = *reinterpret_cast<const float4*>(&slots[which][parity][w]);
            t += (s.x + s.y) + (s.z + s.w);
        }
        return t;
    }
    __device__ __forceinline__ float one(float v)
    {
        if constexpr (L > 0) {
            return lanes_sum<L>(v);
        } else {
            v = lanes_sum<64>(v);
            if ((threadIdx.x & 63) == 0) slots[0][parity][threadIdx.x >> 6] = v;
            __syncthreads();
            v = total(0);
            parity ^= 1;
            return v;
        }
    }
    __device__ __forceinline__ void two(float& u, float& v)
    {
        if constexpr (L > 0) {
            u = lanes_sum<L>(u);
            v = lanes_sum<L>(v);
        } else {
            u = lanes_sum<64>(u);
            v = lanes_sum<64>(v);
            if ((threadIdx.x & 63) == 0) {
                slots[0][parity][threadIdx.x >> 6] = u;
                slots[1][parity][threadIdx.x >> 6] = v;
            }
            __syncthreads();
            u = total(0);
            v = total(1);
            parity ^= 1;
        }
    }
};

// A lane's part of a row: VPT vectors of 8 channels from channel at[i] on, of
// which the first skip[i] are another lane's (8: all of them, and `at` is of no
// use).
template <int VPT>
struct Part {
    uint32_t at[VPT];
    int skip[VPT];
    bool exact;  // every lane holds whole vectors of its own (uniform)
    __device__ __forceinline__ Part(int C, int lanes, int lane)
    {
        exact = C == lanes * VPT * kVec;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int want = (i * lanes + lane) * kVec, from = min(want, C - kVec);
            skip[i] = min(want - from, kVec);
            at[i] = skip[i] < kVec ? from : kOutside / 8;
        }
    }
    // Byte offset of vector i in rows of T, `sub` values behind the first.
    template <typename T>
    __device__ __forceinline__ uint32_t off(int i, uint32_t sub) const
    {
        return skip[i] < kVec ? (at[i] + sub) * static_cast<uint32_t>(sizeof(T)) : kOutside;
    }
};
template <int VPT>
using Row = float[VPT][kVec];

template <typename T, int VPT>
__device__ __forceinline__ void load_row(rsrc_t r, const uint32_t (&off)[VPT], Raw<T> (&v)[VPT])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i].load(r, off[i]);
}
template <typename T, int VPT>
__device__ __forceinline__ void load_param(const void* p, const Part<VPT>& part, float other, Raw<T> (&v)[VPT])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        v[i].fill(other);
        if (p) v[i].load(rows_from<T>(p, 0), part.template off<T>(i, 0));
    }
}
// A parameter's values for a lane's channels: kept over the rows with one
// vector a lane, in registers or (SHELF, bf16) in the lane's own 16 bytes of
// LDS; read again for each row with two.
template <typename T, int VPT, bool SHELF = false>
struct Param {
    static constexpr bool kKept = VPT == 1 && !SHELF;
    Raw<T> raw[kKept ? VPT : 1];
    const void* p;
    float other;
    uint4* shelf;
    __device__ __forceinline__ Param(const void* from, const Part<VPT>& part, float fill, uint4* own = nullptr) : p(from), other(fill), shelf(own)
    {
        if constexpr (kKept) load_param(p, part, other, raw);
        if constexpr (SHELF) {
            Raw<T> now[VPT];
            load_param(p, part, other, now);
            *shelf = now[0].u[0];
        }
    }
    __device__ __forceinline__ void stay()
    {
        if constexpr (kKept) raw[0].stay();
    }
    __device__ __forceinline__ void get(const Part<VPT>& part, Row<VPT>& v) const
    {
        if constexpr (SHELF) {
            Raw<T> now;
            now.u[0] = *shelf;
            now.get(v[0]);
        } else if constexpr (kKept) {
            raw[0].get(v[0]);
        } else {
            Raw<T> now[VPT];
            load_param(p, part, other, now);
#pragma unroll
            for (int i = 0; i < VPT; ++i) now[i].get(v[i]);
        }
    }
};
template <typename T, int VPT>
__device__ __forceinline__ void get_row(const Raw<T> (&r)[VPT], Row<VPT>& v)
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i].get(v[i]);
}
template <typename T, int VPT>
__device__ __forceinline__ void store_row(rsrc_t r, const uint32_t (&off)[VPT], const Row<VPT>& v)
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) store8<T>(r, off[i], v[i]);
}
#define CONVMI_EACH(i, e)              \
    _Pragma("unroll") for (int i = 0; i < VPT; ++i) _Pragma("unroll") for (int e = 0; e < kVec; ++e)

// A row's own channels of `term`, added up over the lane.
template <int VPT, typename F>
__device__ __forceinline__ float lane_sum(const Part<VPT>& part, F term)
{
    float t = 0.f;
    if (part.exact) {
        CONVMI_EACH(i, e) t += term(i, e);
    } else {
        CONVMI_EACH(i, e) t += e >= part.skip[i] ? term(i, e) : 0.f;
    }
    return t;
}

// Normalises a row in place; its mean (layer) and r.
struct Stats {
    float mean, r;
};
template <int L, int VPT>
__device__ __forceinline__ Stats normalise(int kind, const Part<VPT>& part, float inv_c, float eps, RowSum<L>& rs, Row<VPT>& v)
{
    float mean = 0.f;
    if (kind == kNormLayer) {
        mean = rs.one(lane_sum(part, [&](int i, int e) { return v[i][e]; })) * inv_c;
        CONVMI_EACH(i, e) v[i][e] -= mean;
    }
    const float r = 1.0f / sqrtf(rs.one(lane_sum(part, [&](int i, int e) { return v[i][e] * v[i][e]; })) * inv_c + eps);
    CONVMI_EACH(i, e) v[i][e] *= r;
    return {mean, r};
}

struct NormGrid {
    FastDiv gate;       // division by gate_rows
    int64_t per;        // forward: consecutive rows of a group of lanes, or of a workgroup
};

// L lanes a row, or (L 0) a workgroup of up to MAXT threads.
template <typename T, int VPT, int L, int MAXT>
__global__ __launch_bounds__(MAXT, 4) void norm_fwd_kernel(NormArgs k, NormGrid grid)
{
    __shared__ __align__(16) float slots[2][2][kMaxWaves];
    RowSum<L> rs{slots, 0};
    if (!L) {
        if (threadIdx.x < 4 * kMaxWaves) (&slots[0][0][0])[threadIdx.x] = 0.f;
        __syncthreads();
    }
    const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x;
    const Part<VPT> part(k.C, lanes, lane);
    const float inv_c = 1.0f / k.C;
    const bool each = k.z && k.gate_rows == 1;  // a gate for every element
    Param<T, VPT> post_w(k.post_w, part, 1.f), post_b(k.post_b, part, 0.f), pre_w(k.pre_w, part, 1.f), pre_b(k.pre_b, part, 0.f), s(k.s, part, 1.f);
    constexpr bool kAhead = VPT == 1;  // a row's loads go out before the row before it is worked on

    // A wave's rows follow each other: the 64 / L rows that it takes at a time
    // are neighbours, and so are those it takes next.
    constexpr int R = L ? 64 / L : 1;
    const int sub = L ? (threadIdx.x & 63) / (L ? L : 64) : 0;
    const int wave = L ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const RowWalk walk(L ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x, R, grid.per, k.rows);
    uint32_t off[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) off[i] = part.template off<T>(i, sub * static_cast<uint32_t>(k.C));
    Raw<T> xr[VPT], fr[VPT], zr[VPT];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        if (!walk.has(r, sub)) return;
        load_row(rows_from<T>(k.x, r * k.C), off, xr);
        if (k.f) load_row(rows_from<T>(k.f, r * k.C), off, fr);
        if (each) load_row(rows_from<T>(k.z, r * k.C), off, zr);
    };
    if (kAhead) fetch(walk.first);
    Row<VPT> g;  // s act(z)
    s.get(part, g);
    int64_t gate_at = -1;
    for (int64_t r = walk.first; walk.has(r, sub); r += R) {  // rows r to r + R - 1, as far as they exist
        Row<VPT> v, n, w, b;
        post_w.stay(), post_b.stay(), pre_w.stay(), pre_b.stay(), s.stay();
        if (!kAhead) fetch(r);
        get_row(xr, v);
        if (k.f) get_row(fr, n);
        if (k.z) {
            const int64_t at = each ? r : fdiv(static_cast<uint32_t>(r + sub), grid.gate);
            if (each || at != gate_at) {
                gate_at = at;
                if (!each) {
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (part.skip[i] < kVec) {
                            const T* p = static_cast<const T*>(k.z) + at * k.C + part.at[i];
#pragma unroll
                            for (int h = 0; h < Raw<T>::kWords; ++h) zr[i].u[h] = load16_any(p + h * 4);
                        }
                }
                s.get(part, g);
                get_row(zr, w);
                with_act(k.act, [&](auto kind) __attribute__((always_inline)) { CONVMI_EACH(i, e) g[i][e] *= act_value<kind()>(w[i][e]); });
            }
        }
        if (kAhead) fetch(r + R);
        if (k.f) {
            if (k.post != kNormNone) {
                normalise(k.post, part, inv_c, k.eps, rs, n);
                post_w.get(part, w);
                post_b.get(part, b);
                CONVMI_EACH(i, e) n[i][e] = n[i][e] * w[i][e] + b[i][e];
            }
            CONVMI_EACH(i, e) v[i][e] += g[i][e] * n[i][e];
        }
        if (k.y) store_row<T>(rows_from<T>(k.y, r * k.C), off, v);
        if (k.a) {
            normalise(k.pre, part, inv_c, k.eps, rs, v);
            pre_w.get(part, w);
            pre_b.get(part, b);
            CONVMI_EACH(i, e) v[i][e] = v[i][e] * w[i][e] + b[i][e];
            store_row<T>(rows_from<T>(k.a, r * k.C), off, v);
        }
    }
}

// Threads of the workgroup that takes a row of more than 512 channels, and of
// the gradient's for any.
int row_threads(int C) { return C <= 4096 ? (C + 511) / 512 * 64 : (C + 1023) / 1024 * 64; }
int bwd_threads(int C) { return C <= 512 ? 256 : row_threads(C); }

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
bool sums_apart(int C);
// Pieces wanted where the device holds `hold` workgroups at once: one each, so
// that all end together; fewer where a piece would have too few rows to pay for
// its partial sums, four a CU (or sixteen waves) at most.  Forward and gradient,
// 1024 pieces against as many as are held: 16384 x 4096 bf16 rms norms 405 and
// 388 us, layer norms 490 and 463; 2000 x 3001 fp32 88 and 63; but 9000 x 1500
// bf16 layer norms, of which four workgroups a CU are held, 102 with 1024, 119
// with 512.
int64_t want_pieces(int64_t rows, int C, int64_t hold)
{
    if (sums_apart(C)) return std::max<int64_t>(1, std::min<int64_t>(std::max(1, 1024 / ((C + 2047) / 2048)), rows / 4));
    const int64_t cus = device_cu_count(), most = std::min<int64_t>(4 * cus, cus * 1024 / bwd_threads(C));
    return std::max<int64_t>(1, std::min(std::min(hold, most), rows / (C <= 512 ? 8 : 2)));
}
Pieces make_pieces(int64_t rows, int64_t gate_rows, bool has_gate, int64_t want)
{
    Pieces p{};
    const bool shared = has_gate && gate_rows > 1;
    p.group = shared ? gate_rows : std::max<int64_t>(rows, 1);
    const int64_t groups = rows / p.group;
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

// Waves of a SIMD: four where the registers hold a row of bf16, its parameters
// and the gate's slope being in LDS then (its lane's own places: no barrier);
// two where the biases' sums, fp32 rows or a second vector a lane would spill.
// 16384 x 4096 bf16, gradient: 240 us with the shelf; 290 with the parameters
// in registers, where 56 spills made 300 MB of the 1.4 GB; 310 with two waves.
// 8192 x 2048 with a shared gate, forward and gradient: 81 us with four waves,
// 92 with two.
template <typename T, int VPT, int L, bool MORE>
constexpr bool bwd_shelf() { return sizeof(T) == 2 && VPT == 1 && !MORE && !L; }
template <typename T, int VPT, int L, bool MORE>
constexpr int bwd_waves() { return bwd_shelf<T, VPT, L, MORE>() ? 4 : 2; }
// BIAS: with the sums of a layer norm's biases.  SHARED: a gate row serves
// several rows.  Without SUMS, for rows whose sums do not fit in the registers
// beside them: the rows alone, and their statistics.
template <typename T, int VPT, int L, int MAXT, bool BIAS, bool SHARED, bool SUMS>
__global__ __launch_bounds__(MAXT, (MAXT > 512 ? 4 : bwd_waves<T, VPT, L, BIAS>())) void norm_bwd_kernel(NormArgs k, Pieces pc, FastDiv gate_rows)
{
    __shared__ __align__(16) float slots[2][2][kMaxWaves];
    __shared__ float joined[L ? 4 : 1][L ? 64 * VPT * kVec : 1];
    RowSum<L> rs{slots, 0};
    if (!L) {
        if (threadIdx.x < 4 * kMaxWaves) (&slots[0][0][0])[threadIdx.x] = 0.f;
        __syncthreads();
    }
    constexpr int R = L ? 64 / L : 1;  // rows of a wave at a time
    const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x;
    const int wave = L ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0, sub = L ? (threadIdx.x & 63) / (L ? L : 64) : 0;
    const Part<VPT> part(k.C, lanes, lane);
    const float inv_c = 1.0f / k.C;
    static_assert(SUMS || (!L && !SHARED && !BIAS), "");
    const bool each = !SHARED && k.z;
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * kSums * k.C;  // in k.part
    uint32_t off[VPT], param_off[VPT], sum_off[VPT];  // in rows, in one row, in a row of fp32
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        off[i] = part.template off<T>(i, sub * static_cast<uint32_t>(k.C));
        param_off[i] = part.template off<T>(i, 0);
        sum_off[i] = part.template off<float>(i, 0);
    }
    constexpr bool kShelf = bwd_shelf<T, VPT, L, BIAS>();
    __shared__ uint4 shelf[kShelf ? 4 : 1][kShelf ? MAXT : 1];
    const int own = kShelf ? threadIdx.x : 0;
    Param<T, VPT, kShelf> post_w(k.post_w, part, 1.f, &shelf[0][own]), post_b(k.post_b, part, 0.f, &shelf[kShelf ? 1 : 0][own]),
        pre_w(k.pre_w, part, 1.f, &shelf[kShelf ? 2 : 0][own]), s(k.s, part, 1.f, &shelf[kShelf ? 3 : 0][own]);
    __shared__ float4 slopes[2][kShelf ? MAXT : 1];  // a lane's act'(z)
    constexpr bool kAhead = VPT == 1;  // a row's loads go out before the row before it is worked on

    // In the order of the partial rows; for a shared gate [kSumScale] is the
    // group's sum of P, from which dz and the group's part of ds follow.
    constexpr int NS = !SUMS ? 1 : BIAS ? kSumGate : 3;
    float sum[NS][VPT][kVec], scale_sum[SHARED ? VPT : 1][kVec];
#pragma unroll
    for (int q = 0; q < NS; ++q) CONVMI_EACH(i, e) sum[q][i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < (SHARED ? VPT : 1); ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) scale_sum[i][e] = 0.f;

    // Adds a column sum over the groups of lanes of the workgroup (in order)
    // and lets `put` have it, in the first one's lanes.
    auto join = [&](Row<VPT>& v, auto put) __attribute__((always_inline)) {
        if constexpr (L > 0) {
            CONVMI_EACH(i, e)
            {
                if (L <= 8) v[i][e] += __shfl_xor(v[i][e], 8);
                if (L <= 16) v[i][e] += __shfl_xor(v[i][e], 16);
                if (L <= 32) v[i][e] += __shfl_xor(v[i][e], 32);
            }
            __syncthreads();
            if (sub == 0) CONVMI_EACH(i, e) joined[wave][(i * kVec + e) * L + lane] = v[i][e];
            __syncthreads();
            if (wave == 0 && sub == 0) {
                CONVMI_EACH(i, e)
                {
                    const int at = (i * kVec + e) * L + lane;
                    v[i][e] = ((joined[0][at] + joined[1][at]) + joined[2][at]) + joined[3][at];
                }
                put(v);
            }
        } else {
            put(v);
        }
    };

    const int64_t group0 = pc.split > 1 ? blockIdx.x / pc.split : blockIdx.x * pc.groups;
    int64_t r0 = SUMS ? group0 * pc.group + (pc.split > 1 ? (blockIdx.x % pc.split) * pc.per : 0) : blockIdx.x;
    const int64_t end = SUMS ? min(pc.split > 1 ? (group0 + 1) * pc.group : k.rows, r0 + pc.per) : k.rows;
    const int64_t step = L ? 4 * R : SUMS ? 1 : gridDim.x;
    Raw<T> xr[VPT], fr[VPT], zr[VPT], yr[VPT], ar[VPT];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        load_row(rows_from<T>(k.x, r * k.C), off, xr);
        if (k.f) load_row(rows_from<T>(k.f, r * k.C), off, fr);
        if (each) load_row(rows_from<T>(k.z, (SUMS ? r : fdiv(static_cast<uint32_t>(r), gate_rows)) * static_cast<int64_t>(k.C)), off, zr);
    };
    auto fetch_grads = [&](int64_t r) __attribute__((always_inline)) {
        if (k.dy) load_row(rows_from<T>(k.dy, r * k.C), off, yr);
        if (k.da) load_row(rows_from<T>(k.da, r * k.C), off, ar);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) yr[i].fill(0.f);
    while (r0 < end) {
        const int64_t stop = SHARED ? min(end, (r0 / pc.group + 1) * pc.group) : end;
        const int64_t begin = r0 + wave * R;
        if (kAhead && sub < stop - begin) {
            fetch(begin);
            fetch_grads(begin);
        }
        Row<VPT> zv, zd;  // act(z) and its derivative
        CONVMI_EACH(i, e) zv[i][e] = 1.f, zd[i][e] = 0.f;
        auto gate = [&]() __attribute__((always_inline)) {
            get_row(zr, zv);
            with_act(k.act, [&](auto kind) __attribute__((always_inline)) {
                CONVMI_EACH(i, e)
                {
                    const ActPair p = act_pair<kind()>(zv[i][e]);
                    zv[i][e] = p.v;
                    zd[i][e] = p.d;
                }
            });
            if constexpr (kShelf) {
                slopes[0][own] = make_float4(zd[0][0], zd[0][1], zd[0][2], zd[0][3]);
                slopes[1][own] = make_float4(zd[0][4], zd[0][5], zd[0][6], zd[0][7]);
            }
        };
        if (SHARED) {
            load_row(rows_from<T>(k.z, r0 / pc.group * k.C), param_off, zr);
            gate();
        }
        for (int64_t r = begin; r < stop; r += step) {  // rows r to r + R - 1
            if (sub >= stop - r) break;
            const bool more = kAhead && sub < stop - r - step;
            Row<VPT> v, n, d, w, b;
            Stats sf{0.f, 1.f}, sy{0.f, 1.f};
            float c1 = 0.f, c2 = 0.f;
            auto stay = [&]() __attribute__((always_inline)) {
                post_w.stay(), post_b.stay(), pre_w.stay(), s.stay();
            };
            stay();
            if (!kAhead) fetch(r);
            get_row(xr, v);
            if (k.f) get_row(fr, n);
            if (each) gate();
            if (more) fetch(r + step);
            // y again: v, with fh in n
            if (k.f) {
                if (k.post != kNormNone) sf = normalise(k.post, part, inv_c, k.eps, rs, n);
                Row<VPT> g;
                s.get(part, g);
                post_w.get(part, w);
                post_b.get(part, b);
                CONVMI_EACH(i, e) v[i][e] += g[i][e] * zv[i][e] * (n[i][e] * w[i][e] + b[i][e]);
            }
            if (k.da) sy = normalise(k.pre, part, inv_c, k.eps, rs, v);
            // D in d
            if (!kAhead) fetch_grads(r);
            get_row(yr, d);
            if (k.da) {
                Row<VPT> t;
                get_row(ar, t);
                pre_w.get(part, w);
                CONVMI_EACH(i, e)
                {
                    if constexpr (SUMS) sum[kSumPreW][i][e] += t[i][e] * v[i][e];
                    if constexpr (BIAS) sum[kSumPreB][i][e] += t[i][e];
                    t[i][e] *= w[i][e];
                }
                if (more) fetch_grads(r + step);
                c1 = lane_sum(part, [&](int i, int e) { return t[i][e]; });
                c2 = lane_sum(part, [&](int i, int e) { return t[i][e] * v[i][e]; });
                rs.two(c1, c2);
                c1 = k.pre == kNormLayer ? c1 * inv_c : 0.f;
                c2 *= inv_c;
                CONVMI_EACH(i, e) d[i][e] += sy.r * (t[i][e] - c1 - v[i][e] * c2);
            } else if (more) {
                fetch_grads(r + step);
            }
            if (k.dx) store_row<T>(rows_from<T>(k.dx, r * k.C), off, d);
            if (!SUMS && threadIdx.x == 0) k.stats[r] = RowStats{sf.mean, sf.r, sy.mean, sy.r, c1, c2};
            if (!k.f) continue;
            // gate, scale and branch: fh in n, D in d; v is free
            stay();
            post_w.get(part, w);
            post_b.get(part, b);
            CONVMI_EACH(i, e) v[i][e] = d[i][e] * (n[i][e] * w[i][e] + b[i][e]);  // P
            Row<VPT> g;
            s.get(part, g);
            if constexpr (SUMS) CONVMI_EACH(i, e) sum[kSumScale][i][e] += SHARED ? v[i][e] : v[i][e] * zv[i][e];
            if (each && k.dz && (SUMS || k.gate_rows == 1)) {
                if constexpr (kShelf) {
                    const float4 lo = slopes[0][own], hi = slopes[1][own];
                    const float slope[kVec] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    CONVMI_EACH(i, e) v[i][e] *= g[i][e] * slope[e];
                } else {
                    CONVMI_EACH(i, e) v[i][e] *= g[i][e] * zd[i][e];
                }
                store_row<T>(rows_from<T>(k.dz, r * k.C), off, v);
            }
            CONVMI_EACH(i, e)
            {
                const float dn = d[i][e] * (g[i][e] * zv[i][e]);
                if constexpr (SUMS) sum[kSumPostW][i][e] += dn * n[i][e];
                if constexpr (BIAS) sum[kSumPostB][i][e] += dn;
                v[i][e] = dn * w[i][e];  // without a post norm w is 1
            }
            if (k.post != kNormNone) {
                float e1 = lane_sum(part, [&](int i, int e) { return v[i][e]; });
                float e2 = lane_sum(part, [&](int i, int e) { return v[i][e] * n[i][e]; });
                rs.two(e1, e2);
                e1 = k.post == kNormLayer ? e1 * inv_c : 0.f;
                e2 *= inv_c;
                CONVMI_EACH(i, e) v[i][e] = sf.r * (v[i][e] - e1 - n[i][e] * e2);
            }
            if (k.df) store_row<T>(rows_from<T>(k.df, r * k.C), off, v);
        }
        if constexpr (SHARED) {
            Row<VPT> g, t;
            s.get(part, g);
            CONVMI_EACH(i, e)
            {
                t[i][e] = sum[kSumScale][i][e] * g[i][e] * zd[i][e];
                scale_sum[i][e] += sum[kSumScale][i][e] * zv[i][e];
                sum[kSumScale][i][e] = 0.f;
            }
            // the group is whole here (split 1): its gate row's gradient is done
            const int64_t group = r0 / pc.group;
            join(t, [&](Row<VPT>& v) {
                if (pc.split > 1) store_row<float>(rows_from<float>(k.part, mine + kSumGate * k.C), sum_off, v);
                else if (k.dz) store_row<T>(rows_from<T>(k.dz, group * k.C), param_off, v);
            });
        }
        r0 = stop;
    }
    if constexpr (SHARED) CONVMI_EACH(i, e) sum[kSumScale][i][e] = scale_sum[i][e];
#pragma unroll
    for (int q = 0; q < (SUMS ? NS : 0); ++q)
        join(sum[q], [&](Row<VPT>& v) { store_row<float>(rows_from<float>(k.part, mine + static_cast<int64_t>(q) * k.C), sum_off, v); });
}
#undef CONVMI_EACH

// Rows too long for the registers, or shorter than a vector: a workgroup walks
// a row several times, whatever its length; later passes find it in the caches.
constexpr int kLongThreads = 512;
struct LongRow {
    const NormArgs& k;
    float inv_c;
    RowSum<0> rs;
    template <typename F>
    __device__ __forceinline__ float sum(F term)
    {
        float t = 0.f;
        for (int c = threadIdx.x; c < k.C; c += kLongThreads) t += term(c);
        return rs.one(t);
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
    __shared__ __align__(16) float slots[2][2][kMaxWaves];
    if (threadIdx.x < 4 * kMaxWaves) (&slots[0][0][0])[threadIdx.x] = 0.f;
    __syncthreads();
    LongRow row{k, 1.0f / k.C, RowSum<0>{slots, 0}};
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

// The same walk for the gradient's rows.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_bwd_long_kernel(NormArgs k)
{
    __shared__ __align__(16) float slots[2][2][kMaxWaves];
    if (threadIdx.x < 4 * kMaxWaves) (&slots[0][0][0])[threadIdx.x] = 0.f;
    __syncthreads();
    LongRow row{k, 1.0f / k.C, RowSum<0>{slots, 0}};
    for (int64_t r = blockIdx.x; r < k.rows; r += gridDim.x) {
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
        if (threadIdx.x == 0) k.stats[r] = RowStats{fm, fr, ym, yr, c1, c2};
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
            if (k.dx) store_f(static_cast<T*>(k.dx) + r * k.C + c, d);
            if (!f) continue;
            if (z && k.dz && k.gate_rows == 1)
                store_f(static_cast<T*>(k.dz) + r * k.C + c, d * branch(c) * param<T>(k.s, c, 1.f) * act_pair(k.act, load_f(z + c)).d);
            if (k.df) {
                const float dn = d * factor(c);
                const float t = k.post == kNormNone ? dn : fr * (dn * param<T>(k.post_w, c, 1.f) - e1 - fh(c) * e2);
                store_f(static_cast<T*>(k.df) + r * k.C + c, t);
            }
        }
    }
}

// The column sums of rows that were worked on without them, from their
// statistics: a second stream over dy, da, x, f and z, in which a lane owns V
// columns of a piece of the rows and nothing crosses lanes.  975 x 11823 bf16,
// layer norms, a full gate, forward and gradient: 202 us; 652 with the sums in
// the first pass, whose registers then spill.
template <typename T, int V>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs k, Pieces pc)
{
    const int want = (blockIdx.x * 256 + threadIdx.x) * V;
    if (want >= k.C) return;
    const int c = min(want, k.C - V);  // the last lane repeats columns of the one before: the same sums
    const bool shared = k.z && k.gate_rows > 1;
    auto get = [&](const void* p, int64_t row, float (&v)[V]) __attribute__((always_inline)) {
        const T* t = static_cast<const T*>(p) + row * k.C + c;
        if constexpr (V == 1) {
            v[0] = load_f(t);
        } else {
            Raw<T> r;
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords; ++i) r.u[i] = load16_any(t + i * 4);
            r.get(v);
        }
    };
    float post_w[V], post_b[V], pre_w[V], s[V], sum[kSums][V], zv[V], zd[V];
#pragma unroll
    for (int e = 0; e < V; ++e) post_w[e] = pre_w[e] = s[e] = zv[e] = 1.f, post_b[e] = zd[e] = 0.f;
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[q][e] = 0.f;
    if (k.post_w) get(k.post_w, 0, post_w);
    if (k.post_b) get(k.post_b, 0, post_b);
    if (k.pre_w) get(k.pre_w, 0, pre_w);
    if (k.s) get(k.s, 0, s);
    const int piece = blockIdx.y;
    const int64_t group0 = pc.split > 1 ? piece / pc.split : piece * pc.groups;
    int64_t r0 = group0 * pc.group + (pc.split > 1 ? (piece % pc.split) * pc.per : 0);
    const int64_t end = min(pc.split > 1 ? (group0 + 1) * pc.group : k.rows, r0 + pc.per);
    float* mine = k.part + static_cast<int64_t>(piece) * kSums * k.C + c;
    auto gate = [&](int64_t row) __attribute__((always_inline)) {
        get(k.z, row, zv);
        with_act(k.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const ActPair p = act_pair<kind()>(zv[e]);
                zv[e] = p.v;
                zd[e] = p.d;
            }
        });
    };
    while (r0 < end) {
        const int64_t stop = shared ? min(end, (r0 / pc.group + 1) * pc.group) : end;
        if (shared) gate(r0 / pc.group);
        float P[V];  // the group's sum
#pragma unroll
        for (int e = 0; e < V; ++e) P[e] = 0.f;
#pragma unroll 2
        for (int64_t r = r0; r < stop; ++r) {
            const RowStats t = k.stats[r];
            float d[V], q[V], v[V], n[V];
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = q[e] = n[e] = 0.f;
            get(k.x, r, v);
            if (k.f) get(k.f, r, n);
            if (k.dy) get(k.dy, r, d);
            if (k.da) get(k.da, r, q);
            if (k.z && !shared) gate(r);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float fh = k.post != kNormNone ? (n[e] - t.f_mean) * t.f_r : n[e];
                const float branch = fh * post_w[e] + post_b[e], factor = s[e] * zv[e];
                if (k.da) {
                    const float yh = ((k.f ? v[e] + factor * branch : v[e]) - t.y_mean) * t.y_r;
                    sum[kSumPreW][e] += q[e] * yh;
                    sum[kSumPreB][e] += q[e];
                    d[e] += t.y_r * (q[e] * pre_w[e] - t.c1 - yh * t.c2);
                }
                const float p = d[e] * branch, dn = d[e] * factor;
                if (shared) P[e] += p;
                else sum[kSumScale][e] += p * zv[e];
                sum[kSumPostW][e] += dn * fh;
                sum[kSumPostB][e] += dn;
            }
        }
        if (shared) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sum[kSumScale][e] += P[e] * zv[e];
                const float g = P[e] * s[e] * zd[e];
                if (pc.split > 1) mine[static_cast<int64_t>(kSumGate) * k.C + e] = g;
                else if (k.dz) store_f(static_cast<T*>(k.dz) + r0 / pc.group * k.C + c + e, g);
            }
        }
        r0 = stop;
    }
#pragma unroll
    for (int q = 0; q < kSumGate; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) mine[static_cast<int64_t>(q) * k.C + e] = sum[q][e];
}

// Rows of up to this many channels stay in the registers of a workgroup, and of
// up to this many with their column sums.
constexpr int kRegisterRow = 16384, kSumRow = 8192;
bool sums_apart(int C) { return C > kSumRow || C < kVec; }

// Calls f with the vectors of a lane, the lanes of a row (0: a workgroup) and
// the threads of its limit.  Rows of a wave use as many lanes as they have
// vectors; longer ones a workgroup, two vectors a lane past 4096 channels (2000 x
// 6000 fp32 layer norms, forward and gradient: 239 us; 308 with one vector and
// twice the threads, whose halved registers spill).
template <typename F>
void with_shape(int C, F f)
{
    const int n = (C + kVec - 1) / kVec;
    typedef std::integral_constant<int, 0> N0;
    typedef std::integral_constant<int, 1> N1;
    typedef std::integral_constant<int, 2> N2;
    typedef std::integral_constant<int, 256> T256;
    if (n <= 8) f(N1{}, std::integral_constant<int, 8>{}, T256{});
    else if (n <= 16) f(N1{}, std::integral_constant<int, 16>{}, T256{});
    else if (n <= 32) f(N1{}, std::integral_constant<int, 32>{}, T256{});
    else if (n <= 64) f(N1{}, std::integral_constant<int, 64>{}, T256{});
    else if (n <= 512) f(N1{}, N0{}, std::integral_constant<int, 512>{});
    else if (n <= 1024) f(N2{}, N0{}, std::integral_constant<int, 512>{});
    else f(N2{}, N0{}, std::integral_constant<int, 1024>{});
}

template <typename T>
hipError_t fwd(const NormArgs& a, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    const int64_t cus = device_cu_count();
    if (a.C > kRegisterRow || a.C < kVec)
        return launch(norm_fwd_long_kernel<T>, dim3(std::min<int64_t>(a.rows, cus * 4)), dim3(kLongThreads), 0, s, a);
    hipError_t e = hipSuccess;
    with_shape(a.C, [&](auto vpt, auto l, auto maxt) {
        NormGrid g;
        g.gate = make_fastdiv(static_cast<uint32_t>(a.gate_rows));
        const int threads = l() ? 256 : row_threads(a.C);
        // rows at a time of a workgroup, and as many workgroups as the device
        // holds at four waves a SIMD
        const int64_t at_once = l() ? 256 / (l() ? l() : 1) : 1;
        const int64_t hold = cus * 16 * 64 / threads;
        g.per = std::max<int64_t>(1, (a.rows + hold * at_once - 1) / (hold * at_once));
        const unsigned grid = static_cast<unsigned>((a.rows + at_once * g.per - 1) / (at_once * g.per));
        e = launch(norm_fwd_kernel<T, vpt(), l(), maxt()>, dim3(grid), dim3(threads), 0, s, a, g);
    });
    return e;
}

// Workgroups of a kernel that the device holds at once.
template <auto KERNEL>
int64_t held(int threads)
{
    static std::atomic<int> known[kMaxWaves + 1];
    std::atomic<int>& at = known[threads / 64];
    int n = at.load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(KERNEL), threads, 0) != hipSuccess || n < 1) n = 1;
        at.store(n, std::memory_order_relaxed);
    }
    return static_cast<int64_t>(n) * device_cu_count();
}

template <typename T>
hipError_t bwd(const NormArgs& given, hipStream_t s)
{
    NormArgs a = given;
    const bool shared = a.z && a.gate_rows > 1;
    const bool bias = a.dpre_b || a.dpost_b;
    typedef void (*Kernel)(NormArgs, Pieces, FastDiv);
    Kernel kernel = nullptr;  // rows and sums in one
    int64_t hold = 0;
    if (!sums_apart(a.C))
        with_shape(a.C, [&](auto vpt, auto l, auto maxt) {
            if constexpr (maxt() < 1024) {
                auto take = [&](auto b, auto sh) {
                    kernel = norm_bwd_kernel<T, vpt(), l(), maxt(), b(), sh(), true>;
                    hold = held<norm_bwd_kernel<T, vpt(), l(), maxt(), b(), sh(), true>>(bwd_threads(a.C));
                };
                if (bias) shared ? take(std::true_type{}, std::true_type{}) : take(std::true_type{}, std::false_type{});
                else shared ? take(std::false_type{}, std::true_type{}) : take(std::false_type{}, std::false_type{});
            }
        });
    const Pieces pc = make_pieces(a.rows, a.gate_rows, a.z != nullptr, want_pieces(a.rows, a.C, hold));
    a.stats = reinterpret_cast<RowStats*>(a.part + static_cast<int64_t>(pc.count) * kSums * a.C);
    SumArgs sums{};
    const int64_t pitch = static_cast<int64_t>(kSums) * a.C;
    void* out[kSumGate] = {a.dpre_w, a.dpost_w, a.ds, a.dpre_b, a.dpost_b};
    // whether columns are summed at all, and whether their pieces' sums are added
    bool columns = shared && a.dz && a.rows > 0, added = columns && pc.split > 1;
    if (added) add_sum(sums, a.part + static_cast<int64_t>(kSumGate) * a.C, pitch, a.C, pc.split, a.dz, static_cast<int>(a.rows / pc.group));
    for (int q = 0; q < kSumGate; ++q) {
        add_sum(sums, a.part + static_cast<int64_t>(q) * a.C, pitch, a.C, pc.count, out[q]);
        if (out[q]) columns = added = true;
    }
    CallEvents events;
    hipError_t e = hipSuccess;
    if (pc.count > 0) {
        events.next(sums_apart(a.C) ? !columns : !added);
        const dim3 grid(pc.count);
        const FastDiv gate = make_fastdiv(static_cast<uint32_t>(a.gate_rows));
        if (sums_apart(a.C)) {
            const dim3 rows(static_cast<unsigned>(std::min<int64_t>(a.rows, device_cu_count() * (a.C > kRegisterRow ? 4 : 1))));
            if (a.C > kRegisterRow || a.C < kVec)
                e = launch(norm_bwd_long_kernel<T>, rows, dim3(kLongThreads), 0, s, a);
            else
                e = launch(norm_bwd_kernel<T, 2, 0, 1024, false, false, false>, rows, dim3(row_threads(a.C)), 0, s, a, pc, gate);
            if (e != hipSuccess) return e;
            const unsigned v = a.C < kVec ? 1 : kVec;
            if (columns) {
                events.next(!added);
                e = launch(v == 1 ? norm_columns_kernel<T, 1> : norm_columns_kernel<T, kVec>, dim3((a.C + 256 * v - 1) / (256 * v), pc.count), dim3(256), 0, s, a, pc);
            }
        } else {
            e = launch(kernel, grid, dim3(bwd_threads(a.C)), 0, s, a, pc, gate);
        }
    }
    if (e != hipSuccess || !added) return e;
    events.next(true);
    return launch_sums(sums, sizeof(T) == 2, s);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s)
{
    return dtype ? fwd<bf16_t>(a, s) : fwd<float>(a, s);
}

size_t norm_bwd_workspace(int64_t rows, int C)
{
    if (rows == 0) return 0;
    // for as many pieces as any form of the kernel may have
    const int64_t pieces = want_pieces(rows, C, std::numeric_limits<int64_t>::max());
    return static_cast<size_t>(pieces) * kSums * C * sizeof(float) + (sums_apart(C) ? static_cast<size_t>(rows) * sizeof(RowStats) : 0);
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s)
{
    return dtype ? bwd<bf16_t>(a, s) : bwd<float>(a, s);
}

}  // namespace convmi
