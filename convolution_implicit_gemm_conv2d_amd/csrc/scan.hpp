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

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Lanes whose bit DIST is 0 receive u of themselves and of a partner whose bit
// is 1, the others v: two sums over a pair of lanes for the price of one.  Log2
// of a span such steps sum as many values over its lanes.  The partner is the
// lane at distance DIST; of 4, the mirrored lane of eight, which is as good
// where the steps below follow (MIRROR).
template <int DIST, bool MIRROR>
__device__ __forceinline__ float merge(float u, float v)
{
    if constexpr (DIST == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(u), __float_as_uint(v), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (DIST == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(u), __float_as_uint(v), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
        const bool high = (threadIdx.x & DIST) != 0;
        const float mine = high ? v : u, other = high ? u : v;
        if constexpr (DIST == 8) return mine + dpp_of<0x128>(other);              // row_ror:8
        else if constexpr (DIST == 4 && MIRROR) return mine + dpp_of<0x141>(other);  // row_half_mirror
        else if constexpr (DIST == 4) {  // row_shr:4, row_shl:4: all lanes take part in both
            const float below = dpp_of<0x114>(other), above = dpp_of<0x104>(other);
            return mine + (high ? below : above);
        } else return mine + dpp_of<DIST == 2 ? 0x4e : 0xb1>(other);                // quad_perm
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
            v[0] = merge<FIRST, LAST == 1>(v[0], v[0]);
            merge_all<FIRST / 2, LAST, 1>(v);
        } else {
#pragma unroll
            for (int i = 0; i < K / 2; ++i) v[i] = merge<FIRST, LAST == 1>(v[2 * i], v[2 * i + 1]);
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
    static constexpr int SP = NS == 3 ? 4 : NS, LP = GR * SP;  // a group's and a row's place in LDS: aligned reads
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

// A tile: up to kTile rows, between two multiples of kTile, of a sequence and a
// share.  The rows of the first one of [begin, end), and of the last one; 0 where
// there are none.
__device__ __forceinline__ int rows_from(int begin, int end)
{
    const int left = end - begin, room = kTile - (begin & (kTile - 1));
    return left < room ? left : room;
}
__device__ __forceinline__ int rows_to(int begin, int end)
{
    const int left = end - begin, room = end > begin ? ((end - 1) & (kTile - 1)) + 1 : 0;
    return left < room ? left : room;
}

// One value through a buffer resource; offsets past its end read 0 and write
// nothing, which is all that rows, channels and states that do not exist need.
__device__ __forceinline__ float fetch(rsrc_t r, uint32_t at, float)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}
__device__ __forceinline__ bf16_t fetch(rsrc_t r, uint32_t at, bf16_t) { return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0); }
__device__ __forceinline__ void put(rsrc_t r, uint32_t at, float v, float) { __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), r, at, 0, 0); }
__device__ __forceinline__ void put(rsrc_t r, uint32_t at, float v, bf16_t) { __builtin_amdgcn_raw_buffer_store_b16(f_to_bf16(v), r, at, 0, 0); }

// This lane's values of a tensor of rows: rows l.row, l.row + GR, ... of a tile.
// The tensor is walked tile by tile: `at` is the next tile's first row (going
// up) or the one behind its last (going down).
template <typename T, int GR, int NS>
struct Rows {
    typedef Lanes<GR, NS> L;
    const char* at;
    uint32_t stride, off;  // bytes
    __device__ Rows(const L& l, const void* p, int64_t elements, int row0)
        : at(static_cast<const char*>(p) + row0 * elements * static_cast<int64_t>(sizeof(T))), stride(static_cast<uint32_t>(elements) * sizeof(T))
    {
        off = l.on ? static_cast<uint32_t>(l.row) * stride + static_cast<uint32_t>(l.c) * static_cast<uint32_t>(sizeof(T)) : kOutside;
    }
    template <bool UP>
    __device__ rsrc_t tile(int rows)
    {
        const uint32_t bytes = static_cast<uint32_t>(rows) * stride;
        if (!UP) at -= bytes;
        const rsrc_t r = make_rsrc(at, bytes);
        if (UP) at += bytes;
        return r;
    }
    template <bool UP>
    __device__ void load(int rows, T* v)
    {
        const rsrc_t r = tile<UP>(rows);
#pragma unroll
        for (int i = 0; i < L::R; ++i) v[i] = fetch(r, off + i * GR * stride, T());
    }
    template <bool UP>
    __device__ void store(int rows, const float* v)
    {
        const rsrc_t r = tile<UP>(rows);
#pragma unroll
        for (int i = 0; i < L::R; ++i) put(r, off + i * GR * stride, v[i], T());
    }
};

// This lane's states of a [channels, n] array of fp32, through a buffer: whole
// groups of NS states in one access where n is a multiple of NS.
template <int GR, int NS>
struct States {
    uint32_t off;  // bytes
    int have;      // states of this lane
    bool whole;
    __device__ States(const ScanArgs& a, const Lanes<GR, NS>& l)
    {
        have = l.on ? a.n - l.n0 : 0;
        whole = a.n % NS == 0;
        off = have > 0 ? (static_cast<uint32_t>(l.c) * a.n + l.n0) * 4 : kOutside;
    }
    __device__ void put(rsrc_t r, const float* v) const
    {
        if (NS == 2 && whole) {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(decltype(__builtin_amdgcn_raw_buffer_load_b64(r, 0, 0, 0)), make_uint2(__float_as_uint(v[0]), __float_as_uint(v[NS > 1 ? 1 : 0]))), r, off, 0, 0);
        } else if (NS == 4 && whole) {
            buffer_store16(r, off, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[NS > 1 ? 1 : 0]), __float_as_uint(v[NS > 2 ? 2 : 0]), __float_as_uint(v[NS > 3 ? 3 : 0])));
        } else {
#pragma unroll
            for (int j = 0; j < NS; ++j) scan::put(r, j < have ? off + 4 * j : kOutside, v[j], 0.f);
        }
    }
};

// B and C of a tile, in flight to the wave's LDS.
template <typename T, int GR, int NS>
struct Shared {
    typedef Lanes<GR, NS> L;
    const char *at_b, *at_c;  // walked as Rows are
    uint32_t bs, cs, ob, oc;  // bytes
    int at;                   // this lane's place in a tile; -1 for lanes that do not take part

    __device__ Shared(const ScanArgs& a, const L& l, int row0)
        : at_b(static_cast<const char*>(a.B) + (row0 * a.bs + static_cast<int64_t>(l.group) * a.n) * static_cast<int64_t>(sizeof(T))),
          at_c(static_cast<const char*>(a.C) + (row0 * a.cs + static_cast<int64_t>(l.group) * a.n) * static_cast<int64_t>(sizeof(T))), bs(static_cast<uint32_t>(a.bs) * sizeof(T)),
          cs(static_cast<uint32_t>(a.cs) * sizeof(T))
    {
        const int r = l.lane / L::NP, n = l.lane % L::NP;
        at = r < L::ROWS ? r * L::LP + n / NS * L::SP + n % NS : -1;
        const bool on = at >= 0 && n < a.n;
        ob = on ? r * bs + n * static_cast<uint32_t>(sizeof(T)) : kOutside;
        oc = on ? r * cs + n * static_cast<uint32_t>(sizeof(T)) : kOutside;
    }
    template <bool UP>
    __device__ void load(int rows, T* b, T* c)
    {
        const uint32_t nb = static_cast<uint32_t>(rows) * bs, nc = static_cast<uint32_t>(rows) * cs;
        if (!UP) at_b -= nb, at_c -= nc;
        const rsrc_t rb = make_rsrc(at_b, nb), rc = make_rsrc(at_c, nc);
        if (UP) at_b += nb, at_c += nc;
#pragma unroll
        for (int i = 0; i < L::LOADS; ++i) {
            b[i] = fetch(rb, ob + i * L::ROWS * bs, T());
            c[i] = fetch(rc, oc + i * L::ROWS * cs, T());
        }
    }
    __device__ void put(const T* b, const T* c, float* to_b, float* to_c) const
    {
        if (at < 0) return;
#pragma unroll
        for (int i = 0; i < L::LOADS; ++i)
            if ((i + 1) * L::ROWS <= kTile || at + i * L::ROWS * L::LP < kTile * L::LP) {
                to_b[at + i * L::ROWS * L::LP] = load_f(&b[i]);
                to_c[at + i * L::ROWS * L::LP] = load_f(&c[i]);
            }
    }
};

// What kGroup rows' work reads from LDS.  It is read a group ahead: the compiler
// by itself reads just before the use and waits out the latency each time (4 x 4096 rows
// of 4096 channels, 16 states: 451 us so and 399 a group ahead with 4 groups of lanes, 391
// and 380 with 8).
constexpr int kGroup = 4;
template <int NS, int G, typename D>
struct Operands {
    D d[G];
    float b[G][NS], c[G][NS];
};
// LDS accesses do not cross this point, other instructions may.
__device__ __forceinline__ void lds_stays() { __builtin_amdgcn_sched_barrier(0x47f); }

// A barrier of the workgroup for what its waves have in LDS; loads and stores
// of memory stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier_no_fence();
}

// Zeros in the rows [from, to).
template <typename T, int GR, int NS>
__device__ __forceinline__ void clear_rows(const Lanes<GR, NS>& l, void* p, int64_t stride, int64_t from, int64_t to)
{
    for (int64_t r = from + l.grp; r < to; r += GR)
        if (l.on) store_f(static_cast<T*>(p) + r * stride + l.c, 0.f);
}

// ----------------------------------------------------------------- pieces --

// The rows of a sequence (there are fewer than 2^31).
struct Span {
    int begin, end;
};
__device__ __forceinline__ Span span_of(const ScanArgs& a, int s)
{
    if (!a.starts) return {static_cast<int>(s * a.len), static_cast<int>((s + 1) * a.len)};
    // Whatever the offsets hold, the rows are the tensor's.  They are the same
    // for all lanes, which the compiler does not see in what it loads.
    const int rows = static_cast<int>(a.rows);
    int b = __builtin_amdgcn_readfirstlane(a.starts[s]), e = __builtin_amdgcn_readfirstlane(a.starts[s + 1]);
    b = b < 0 ? 0 : b > rows ? rows : b;
    e = e < b ? b : e > rows ? rows : e;
    return {b, e};
}

// The first sequence that has rows from `row` on, or begins there or later.
__device__ __forceinline__ int first_of(const ScanArgs& a, int row)
{
    int lo = 0, hi = a.seqs;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);  // lo + hi may pass 2^31
        const Span s = span_of(a, mid);
        if (s.end > row || s.begin >= row) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// A workgroup's share of the rows: some whole sequences, or a piece of all rows with
// the sequences [first, last) that have rows in it (empty ones count where they lie).
struct Share {
    int begin, end, first, last;
    bool pieces, end_of_all;

    __device__ Share(const ScanArgs& a, int item) : pieces(a.pieces > 0)
    {
        if (!pieces) {
            first = a.seq0 + item * a.walk;
            last = a.seqs - first > a.walk ? first + a.walk : a.seqs;
            begin = span_of(a, first).begin;
            end = span_of(a, last - 1).end;
            end_of_all = last == a.seqs;
            return;
        }
        const int64_t from = static_cast<int64_t>(item) * a.piece_rows, to = from + a.piece_rows;
        begin = static_cast<int>(from);
        end = static_cast<int>(to < a.rows ? to : a.rows);
        end_of_all = item + 1 == a.pieces;
        first = first_of(a, begin);
        last = end_of_all ? a.seqs : first_of(a, end);
        // a sequence that goes on behind this piece has rows in both
        if (!end_of_all && last < a.seqs && span_of(a, last).begin < end) ++last;
    }
};

// The piece of a row.  In 32 bits: a 64-bit division's scalar registers cost the
// gradient 3 % even where no call has pieces.
__device__ __forceinline__ int piece_of(const ScanArgs& a, int row)
{
    return static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(a.piece_rows));
}

// h + 2^(2 t) e.  The whole power leaves fp32's range where the product does not:
// for a state that grows over many pieces (A > 0, or steps below 0) and was 0, or
// tiny, before them, where 0 times an overflow would be no number, or that fades
// from a large one.  Half of it does not: e is multiplied by 2^t twice, by 2^127 at
// most, which takes any normal e there that 2^(2 t) would.
__device__ __forceinline__ float faded(float t, float e, float h)
{
    const float f = exp2_hw(__builtin_fminf(t, 127.0f));
    return __builtin_fmaf(f, f * e, h);
}

// The state that the `count` pieces before a share (DIR -1) leave to its first
// sequence, or the gradient that those behind it (DIR 1) give to its last one:
// what each of them ends with, faded by the pieces between.  Their ends are
// read four at a time: one after the other costs a load's latency a piece (16384 rows of
// 64 channels in 128 pieces, forward and gradient: 151 us, and 132 four at a time).
template <int DIR, int GR, int NS>
__device__ __forceinline__ void inherit(const ScanArgs& a, const Lanes<GR, NS>& l, const float* A, int item, int count, float* h)
{
    constexpr int U = 4;
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    float passed = 0.f;  // half of the sum
    for (int k = 0; k < count; k += U) {
        float e[U][NS], sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = item + DIR * (1 + (k + u < count ? k + u : k));
            l.read(a, a.ends + q * states, e[u]);
            sum[u] = a.sums[static_cast<int64_t>(q) * a.channels + l.c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u >= count) break;
#pragma unroll
            for (int j = 0; j < NS; ++j) h[j] = faded(A[j] * passed, e[u][j], h[j]);
            passed = __builtin_fmaf(0.5f, sum[u], passed);
        }
    }
}

}  // namespace scan
}  // namespace convmi
