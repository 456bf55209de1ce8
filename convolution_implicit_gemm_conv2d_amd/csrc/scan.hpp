// Selective state space scan: arguments, the lanes' layout and the steps that
// its forward pass, its gradient and its token form share.
//
//   d = softplus(delta + bias) (or delta + bias),   a[n] = exp(d A[n]),
//   h[n] = a[n] h[n] + d B[n] x,   y = (sum_n C[n] h[n] + D x) act(z)
//
// for every channel of a sequence, row after row.  A wave holds CH channels and
// all their states: lane = group * CH + channel, GR = 64 / CH groups of NS
// states each.  Sums over the states then stay inside the wave, which walks its
// sequence without a barrier; B and C of a tile of rows, and d and d x, which
// each lane needs of one row and channel, lie in the wave's own LDS.
#pragma once

#include "act.hpp"
#include "kernels.hpp"

namespace convmi {
namespace scan {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = kScanTile;

// ---------------------------------------------------------- lane exchange --

template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_over(float old, float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL, 0xf, BANKS, false));
}

// Lanes whose bit DIST is 0 receive u of themselves and of their partner (the
// lane at distance DIST), the others v: two sums over a pair of lanes for the
// price of one.  Log2 of a span such steps sum as many values over its lanes.
template <int DIST>
__device__ __forceinline__ float merge(float u, float v)
{
    if constexpr (DIST == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(u), __float_as_uint(v), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (DIST == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(u), __float_as_uint(v), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (DIST == 8) {  // row_ror:8
        return dpp_over<0x128, 0x3>(v, u) + dpp_over<0x128, 0xc>(u, v);
    } else if constexpr (DIST == 4) {  // row_shl:4, row_shr:4
        return dpp_over<0x104, 0x5>(v, u) + dpp_over<0x114, 0xa>(u, v);
    } else {
        const bool high = (threadIdx.x & DIST) != 0;
        const float mine = high ? v : u, other = high ? u : v;
        return mine + dpp_over<DIST == 2 ? 0x4e : 0xb1, 0xf>(other, other);  // quad_perm
    }
}

// K values (a power of two) of every lane, summed over the 2 FIRST / LAST lanes
// at distances FIRST down to LAST: v[0 .. max(1, K LAST / (2 FIRST))) of a lane
// then hold the sums of index (register << levels) + the lane's bits, FIRST's as the lowest.
template <int FIRST, int LAST, int K>
__device__ __forceinline__ void merge_all(float* v)
{
    if constexpr (FIRST >= LAST) {
        if constexpr (K == 1) {
            v[0] = merge<FIRST>(v[0], v[0]);
            merge_all<FIRST / 2, LAST, 1>(v);
        } else {
#pragma unroll
            for (int i = 0; i < K / 2; ++i) v[i] = merge<FIRST>(v[2 * i], v[2 * i + 1]);
            merge_all<FIRST / 2, LAST, K / 2>(v);
        }
    }
}

// Orders a wave's own LDS accesses in the compiled code (the LDS unit keeps
// each wave's order).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// --------------------------------------------------------------- softplus --

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|).  log1p(e) is 2 atanh(s),
// s = e / (2 + e) <= 1/3, by its series (the first term left out is 2e-8
// relative): log2(1 + e) would lose the last places of small steps, as steps
// near 0.001 are.
struct Step {
    float v, d;  // value, derivative
};
template <bool DERIVATIVE>
__device__ __forceinline__ Step softplus(float v)
{
    const float e = exp2_hw(-kLog2e * fabsf(v));
    const float s = e * rcp_hw(2.0f + e), z = s * s;
    float p = 1.0f / 13.0f;
    p = __builtin_fmaf(p, z, 1.0f / 11.0f);
    p = __builtin_fmaf(p, z, 1.0f / 9.0f);
    p = __builtin_fmaf(p, z, 1.0f / 7.0f);
    p = __builtin_fmaf(p, z, 1.0f / 5.0f);
    p = __builtin_fmaf(p, z, 1.0f / 3.0f);
    const float t = 2.0f * s;
    Step r{__builtin_fmaxf(v, 0.0f) + __builtin_fmaf(t * z, p, t), 0.0f};
    if constexpr (DERIVATIVE) r.d = (v < 0.0f ? e : 1.0f) * rcp_hw(1.0f + e);
    return r;
}

// ------------------------------------------------------------------ lanes --

template <int GR, int NS>
struct Lanes {
    static constexpr int CH = 64 / GR;        // channels of a wave
    static constexpr int R = kTile / GR;      // rows of a tile that a lane prepares and finishes
    static constexpr int NP = GR * NS;        // states, padded
    static constexpr int ROWS = 64 / NP;      // whole rows of B that a wave loads at once
    static constexpr int LOADS = (kTile + ROWS - 1) / ROWS;
    int lane, wave, ch, grp, row;  // row: of each GR rows the one that is this lane's
    int c, group, n0;              // channel, group of B and C, first state
    bool on;                       // the channel exists

    __device__ Lanes(const ScanArgs& a, uint32_t block)
    {
        lane = threadIdx.x & 63;
        wave = threadIdx.x >> 6;
        ch = lane % CH;
        grp = lane / CH;
        row = 0;
#pragma unroll
        for (int b = 1, to = GR / 2; b < GR; b <<= 1, to >>= 1) row += (grp & b) ? to : 0;
        group = static_cast<int>(block / a.blocks);
        const int in = static_cast<int>(block % a.blocks) * (kWaves * CH) + wave * CH + ch;
        on = in < a.per_group;
        c = group * a.per_group + (on ? in : 0);
        n0 = grp * NS;
    }
    // This lane's states of a [channels, n] array of fp32 (zeros for those that do not exist).
    __device__ void read(const ScanArgs& a, const float* p, float* v) const
    {
        p += static_cast<int64_t>(c) * a.n + n0;
#pragma unroll
        for (int j = 0; j < NS; ++j) v[j] = 0.f;
        if (!on) return;
        if (a.n == NP) {
#pragma unroll
            for (int j = 0; j < NS; ++j) v[j] = p[j];
        } else {
#pragma unroll
            for (int j = 0; j < NS; ++j)
                if (n0 + j < a.n) v[j] = p[j];
        }
    }
    __device__ void write(const ScanArgs& a, float* p, const float* v) const
    {
        if (!on) return;
        p += static_cast<int64_t>(c) * a.n + n0;
        if (a.n == NP) {
#pragma unroll
            for (int j = 0; j < NS; ++j) p[j] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < NS; ++j)
                if (n0 + j < a.n) p[j] = v[j];
        }
    }
};

// B and C of a tile, in flight to the wave's LDS.  Addresses are a base that
// the wave shares and a 32-bit offset of the lane (the strides are below 2^24).
template <typename T, int GR, int NS>
struct Shared {
    typedef Lanes<GR, NS> L;
    T b[L::LOADS], c[L::LOADS];

    __device__ void load(const ScanArgs& a, const L& l, int64_t row0, int rows)
    {
        const T* pb = static_cast<const T*>(a.B) + row0 * a.bs + static_cast<int64_t>(l.group) * a.n;
        const T* pc = static_cast<const T*>(a.C) + row0 * a.cs + static_cast<int64_t>(l.group) * a.n;
        const int r = l.lane / L::NP, n = l.lane % L::NP;
        const uint32_t ob = static_cast<uint32_t>(r) * static_cast<uint32_t>(a.bs) + n, oc = static_cast<uint32_t>(r) * static_cast<uint32_t>(a.cs) + n;
        const int have = r < L::ROWS && n < a.n ? rows - r : 0;
#pragma unroll
        for (int i = 0; i < L::LOADS; ++i) {
            b[i] = c[i] = T(0);
            if (i * L::ROWS < have) {
                b[i] = pb[ob];
                c[i] = pc[oc];
            }
            pb += L::ROWS * a.bs;
            pc += L::ROWS * a.cs;
        }
    }
    __device__ void put(const L& l, float* to_b, float* to_c) const
    {
        const int at = l.lane;  // row * NP + state
#pragma unroll
        for (int i = 0; i < L::LOADS; ++i)
            if (at < L::ROWS * L::NP && at + i * L::ROWS * L::NP < kTile * L::NP) {
                to_b[at + i * L::ROWS * L::NP] = load_f(&b[i]);
                to_c[at + i * L::ROWS * L::NP] = load_f(&c[i]);
            }
    }
};

// This lane's values of a tensor of rows: rows l.row, l.row + GR, ... of a tile.
template <typename T, int GR, int NS>
__device__ __forceinline__ void load_rows(const Lanes<GR, NS>& l, const void* p, int64_t stride, int64_t row0, int rows, T* v)
{
    const T* at = static_cast<const T*>(p) + row0 * stride;
    const uint32_t off = static_cast<uint32_t>(l.row) * static_cast<uint32_t>(stride) + l.c;
    const int have = l.on ? rows - l.row : 0;
#pragma unroll
    for (int i = 0; i < Lanes<GR, NS>::R; ++i) {
        v[i] = T(0);
        if (i * GR < have) v[i] = at[off];
        at += GR * stride;
    }
}
template <typename T, int GR, int NS>
__device__ __forceinline__ void store_rows(const Lanes<GR, NS>& l, void* p, int64_t stride, int64_t row0, int rows, const float* v)
{
    T* at = static_cast<T*>(p) + row0 * stride;
    const uint32_t off = static_cast<uint32_t>(l.row) * static_cast<uint32_t>(stride) + l.c;
    const int have = l.on ? rows - l.row : 0;
#pragma unroll
    for (int i = 0; i < Lanes<GR, NS>::R; ++i) {
        if (i * GR < have) store_f(at + off, v[i]);
        at += GR * stride;
    }
}
// Zeros in the rows [from, to).
template <typename T, int GR, int NS>
__device__ __forceinline__ void clear_rows(const Lanes<GR, NS>& l, void* p, int64_t stride, int64_t from, int64_t to)
{
    for (int64_t r = from + l.grp; r < to; r += GR)
        if (l.on) store_f(static_cast<T*>(p) + r * stride + l.c, 0.f);
}

// A tile ends at the next multiple of kTile rows, or with its sequence.
__device__ __forceinline__ int64_t tile_end(int64_t at, int64_t end)
{
    const int64_t next = (at | (kTile - 1)) + 1;
    return next < end ? next : end;
}

// ----------------------------------------------------------------- pieces --

// The rows of a sequence.
struct Span {
    int64_t begin, end;
};
__device__ __forceinline__ Span span_of(const ScanArgs& a, int s)
{
    if (!a.starts) return {s * a.len, (s + 1) * a.len};
    // whatever the offsets hold, the rows are the tensor's
    int64_t b = a.starts[s], e = a.starts[s + 1];
    b = b < 0 ? 0 : b > a.rows ? a.rows : b;
    e = e < b ? b : e > a.rows ? a.rows : e;
    return {b, e};
}

// The first sequence that has rows from `row` on, or begins there or later.
__device__ __forceinline__ int first_of(const ScanArgs& a, int64_t row)
{
    int lo = 0, hi = a.seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const Span s = span_of(a, mid);
        if (s.end > row || s.begin >= row) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// A workgroup's share of the rows: one sequence, or a piece of all rows with
// the sequences [first, last) that have rows in it (empty ones count where they lie).
struct Share {
    int64_t begin, end;
    int first, last;
    bool pieces, end_of_all;

    __device__ Share(const ScanArgs& a, int item) : pieces(a.pieces > 0)
    {
        if (!pieces) {
            const Span s = span_of(a, item);
            begin = s.begin;
            end = s.end;
            first = item;
            last = item + 1;
            end_of_all = item + 1 == a.seqs;
            return;
        }
        begin = static_cast<int64_t>(item) * a.piece_rows;
        end = begin + a.piece_rows < a.rows ? begin + a.piece_rows : a.rows;
        end_of_all = item + 1 == a.pieces;
        first = first_of(a, begin);
        last = end_of_all ? a.seqs : first_of(a, end);
        // a sequence that goes on behind this piece has rows in both
        if (!end_of_all && last < a.seqs && span_of(a, last).begin < end) ++last;
    }
};

}  // namespace scan
}  // namespace convmi
