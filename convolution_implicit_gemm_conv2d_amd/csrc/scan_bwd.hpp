// Gradient of the selective scan, for one type: included by the sources that
// build it for bf16 and for fp32.
//
// With G[t] the gradient of h[t] (from y[t] and from h[t + 1]):
//   G[t] = C[t] dy[t] + a[t + 1] G[t + 1],   q[t] = a[t] G[t] h[t - 1],
//   dA = sum_t d q,   dd = sum_n A q + x sum_n B G,   dx = d sum_n B G + D dy,
//   dB = sum_channels d x G,   dC = sum_channels dy h,
// dy being the gradient behind the gate, dz = dout y act'(z).
//
// A tile's states come again from the state in front of it (the forward pass
// keeps one every 16 rows, 4 bytes a state of a row; going back by dividing by a
// would not be stable) and stay in registers, up to two states of a lane factors
// too.  Then the tile goes backwards.  The sums over channels of dB and dC are
// merged over a wave's lanes in pairs, over the workgroup's waves in LDS and
// over workgroups by a kernel of their own: no atomics, so a fixed order.
//
// 8 x 2048 rows of 2048 channels, 16 states, bf16: 563 to 611 us a launch in kernel
// traces (the whole training pass takes 780 to 790 without one), with 835 vector
// instructions of a wave for a tile, which keep the vector units busy 88 % of the
// time; about a third of them are the merges.  Two waves a SIMD (244 registers).
#pragma once

#include "scan.hpp"

namespace convmi {
namespace scan {

constexpr int pow2_of(int v)
{
    int p = 1;
    while (p < v) p *= 2;
    return p;
}
constexpr float kLn2 = 0.69314718055994531f;

// The gradient that a piece passes on to the row before it, from nothing behind
// it, for the pieces in front.
template <typename T, int GR, int NS>
__global__ __launch_bounds__(kThreads) void back_kernel(ScanArgs a)
{
    typedef Lanes<GR, NS> L;
    constexpr int CH = L::CH, R = L::R, LP = L::LP;
    __shared__ float2 lds_d[kWaves][kTile][CH];
    __shared__ float lds_b[kWaves][kTile * LP], lds_c[kWaves][kTile * LP];
    const uint32_t cb = static_cast<uint32_t>(a.groups) * a.blocks;
    const int item = static_cast<int>(blockIdx.x / cb);
    const L l(a, blockIdx.x % cb);
    const Share share(a, item);
    if (share.first >= share.last) return;
    const int s = share.first;
    const Span span = span_of(a, s);
    if (span.begin >= share.begin) return;  // no sequence comes from the piece before
    float2(*dd)[CH] = lds_d[l.wave];
    float *sb = lds_b[l.wave], *sc = lds_c[l.wave];
    float A[NS], g[NS];
    l.read(a, a.A, A);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        A[j] *= kLog2e;
        g[j] = 0.f;
    }
    const float bias = a.bias ? a.bias[l.c] : 0.f;
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    if (span.end <= share.end && a.dlast) l.read(a, a.dlast + s * states, g);
    const int end = span.end < share.end ? span.end : share.end;
    float total = 0.f;
    T dl[R], z[R], dy[R], rb[L::LOADS], rc[L::LOADS];
    Rows<T, GR, NS> rd(l, a.delta, a.ds, end), rz(l, a.z, a.zs, end), rg(l, a.dy, a.channels, end);
    Shared<T, GR, NS> bc(a, l, end);
    auto load = [&](int rows) __attribute__((always_inline)) {
        rd.template load<false>(rows, dl);
        rg.template load<false>(rows, dy);
        rz.template load<false>(a.z ? rows : 0, z);
        bc.template load<false>(rows, rb, rc);
    };
    load(rows_to(share.begin, end));
    for (int to = end; to > share.begin;) {
        const int rows = rows_to(share.begin, to);
        float d[R], dv[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            d[i] = load_f(&dl[i]) + bias;
            if (a.softplus) d[i] = softplus<false>(d[i]).v;
            dv[i] = load_f(&dy[i]);
        }
        if (a.z)
            with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < R; ++i) dv[i] *= act_value<kind()>(load_f(&z[i]));
            });
        wave_fence();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = i * GR + l.row;
            dd[r][l.ch] = make_float2(r < rows ? d[i] : 0.f, r < rows ? dv[i] : 0.f);
        }
        bc.put(rb, rc, sb, sc);
        wave_fence();
        to -= rows;
        load(rows_to(share.begin, to));
#pragma unroll
        for (int r = kTile - 1; r >= 0; --r) {
            const float2 v = dd[r][l.ch];
            const float* c = sc + r * LP + l.grp * L::SP;
            total += v.x;
#pragma unroll
            for (int j = 0; j < NS; ++j) g[j] = __builtin_fmaf(c[j], v.y, g[j]) * exp2_hw(v.x * A[j]);
        }
    }
    l.write(a, a.ends + item * states, g);
    if (l.grp == 0 && l.on) a.sums[static_cast<int64_t>(item) * a.channels + l.c] = total;
}

template <typename T, int GR, int NS>
__global__ __launch_bounds__(kThreads, 2) void bwd_kernel(ScanArgs a)
{
    typedef Lanes<GR, NS> L;
    constexpr int CH = L::CH, R = L::R, NP = L::NP, LP = L::LP;
    constexpr int V = pow2_of(2 * NS);                                   // values of dB and dC a row, padded
    constexpr int RB = CH / V < 1 ? 1 : CH / V > GR ? GR : CH / V;       // rows merged at once
    constexpr int K = V * RB, KEPT = K > CH ? K / CH : 1;
    __shared__ float4 lds_d[kWaves][kTile][CH];
    __shared__ float lds_b[kWaves][kTile * LP], lds_c[kWaves][kTile * LP];
    __shared__ float lds_part[2][kWaves][kTile * 2 * NP];

    const uint32_t cb = static_cast<uint32_t>(a.groups) * a.blocks, block = blockIdx.x % cb;
    const int item = static_cast<int>(blockIdx.x / cb);
    const L l(a, block);
    const Share share(a, item);
    float4(*dd)[CH] = lds_d[l.wave];
    float *sb = lds_b[l.wave], *sc = lds_c[l.wave];
    int mine = 0;  // which of the merged values this lane holds
#pragma unroll
    for (int b = 1, to = CH / 2; b < CH; b <<= 1, to >>= 1) mine += (l.ch & b) ? to : 0;

    float A[NS], g[NS], dA[NS];
    l.read(a, a.A, A);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        A[j] *= kLog2e;
        dA[j] = 0.f;
    }
    const float bias = a.bias ? a.bias[l.c] : 0.f, skip = a.D ? a.D[l.c] : 0.f;
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    float dskip = 0.f, dbias = 0.f;
    int turn = 0;

    for (int s = share.last - 1; s >= share.first; --s) {
        const Span span = span_of(a, s);
#pragma unroll
        for (int j = 0; j < NS; ++j) g[j] = 0.f;
        if (span.end <= share.end) {
            if (a.dlast) l.read(a, a.dlast + s * states, g);
        } else {
            inherit<1>(a, l, A, item, piece_of(a, span.end - 1) - item, g);
        }
        const int begin = span.begin > share.begin ? span.begin : share.begin;
        const int end = span.end < share.end ? span.end : share.end;
        T x[R], dl[R], z[R], dy[R], rb[L::LOADS], rc[L::LOADS];
        float entry[NS];
        Rows<T, GR, NS> rx(l, a.x, a.xs, end), rd(l, a.delta, a.ds, end), rz(l, a.z, a.zs, end), rg(l, a.dy, a.channels, end);
        Rows<T, GR, NS> wx(l, a.dx, a.channels, end), wd(l, a.ddelta, a.channels, end), wz(l, a.dz, a.channels, end);
        Shared<T, GR, NS> bc(a, l, end);
        auto load = [&](int to) __attribute__((always_inline)) {
            const int n = rows_to(begin, to);
            rx.template load<false>(n, x);
            rd.template load<false>(n, dl);
            rg.template load<false>(n, dy);
            rz.template load<false>(a.z ? n : 0, z);
            bc.template load<false>(n, rb, rc);
            // the state in front of the tile; zeros where there is none
            const float* from = to - n > span.begin ? a.saved + static_cast<int64_t>((to - n) / kTile) * states : a.initial ? a.initial + s * states : nullptr;
            const rsrc_t r = make_rsrc(from, from && n > 0 ? static_cast<uint32_t>(states) * 4 : 0);
#pragma unroll
            for (int j = 0; j < NS; ++j) entry[j] = scan::fetch(r, l.on && l.n0 + j < a.n ? (static_cast<uint32_t>(l.c) * a.n + l.n0 + j) * 4 : kOutside, 0.f);
        };
        if (begin < end) load(end);
        for (int to = end; to > begin;) {
            const int rows = rows_to(begin, to);
            // ------------------------------------------ the tile's rows --
            float xf[R], d[R], sig[R], dv[R], dz[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                xf[i] = load_f(&x[i]);
                dz[i] = dv[i] = load_f(&dy[i]);
                const float raw = load_f(&dl[i]) + bias;
                const Step p = softplus<true>(raw);
                d[i] = a.softplus ? p.v : raw;
                sig[i] = a.softplus ? p.d : 1.0f;
            }
            if (a.z)
                with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const ActPair p = act_pair<kind()>(load_f(&z[i]));
                        dz[i] = dv[i] * p.d;
                        dv[i] *= p.v;
                    }
                });
            wave_fence();
#pragma unroll
            for (int i = 0; i < R; ++i) {
                // a row that is not there changes nothing, nor does a channel
                const int r = i * GR + l.row;
                const bool there = r < rows && l.on;
                dd[r][l.ch] = make_float4(there ? d[i] : 0.f, there ? d[i] * xf[i] : 0.f, there ? dv[i] : 0.f, 0.f);
            }
            bc.put(rb, rc, sb, sc);
            wave_fence();
            float first[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) first[j] = entry[j];
            to -= rows;
            load(to);
            // ------------------------------------------- states again --
            constexpr int G = NS <= 2 ? kGroup : 1, NG = kTile / G;  // rows whose operands are read at once
            static_assert(NG % 2 == 0, "operands alternate");
            typedef Operands<NS, G, float4> Ops;
            Ops ops[2];
            auto fetch = [&](Ops& o, int group) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < G; ++r) {
                    o.d[r] = dd[group * G + r][l.ch];
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        o.b[r][j] = sb[(group * G + r) * LP + l.grp * L::SP + j];
                        o.c[r][j] = sc[(group * G + r) * LP + l.grp * L::SP + j];
                    }
                }
            };
            constexpr bool kKeep = NS <= 2;
            float hs[kTile][NS], as[kKeep ? kTile : 1][NS], v[kTile];
            fetch(ops[0], 0);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                fetch(ops[(i + 1) & 1], i + 1 < NG ? i + 1 : NG - 1);  // the last group is also the first one back
                lds_stays();
                const Ops& o = ops[i & 1];
#pragma unroll
                for (int r = 0; r < G; ++r) {
                    const int k = i * G + r;
                    v[k] = 0.f;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const float f = exp2_hw(o.d[r].x * A[j]);
                        if (kKeep) as[kKeep ? k : 0][j] = f;
                        hs[k][j] = __builtin_fmaf(f, k ? hs[k ? k - 1 : 0][j] : first[j], o.d[r].y * o.b[r][j]);
                        v[k] = __builtin_fmaf(hs[k][j], o.c[r][j], v[k]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                merge_all<32, CH, GR>(v + i * GR);
                dz[i] *= __builtin_fmaf(skip, xf[i], v[i * GR]);
            }
            // ------------------------------------------------- and back --
            float* part = lds_part[turn][l.wave];
            float da[NS], ddelta[R], dx[R], w[kTile], u[kTile], m[K];
#pragma unroll
            for (int j = 0; j < NS; ++j) da[j] = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                if (i + 1 < NG) fetch(ops[(i + 1) & 1], NG - 2 - i);
                lds_stays();
                const Ops& o = ops[i & 1];
#pragma unroll
                for (int r = G - 1; r >= 0; --r) {
                    const int k = (NG - 1 - i) * G + r, in = k % RB;
                    w[k] = u[k] = 0.f;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const float e = __builtin_fmaf(o.c[r][j], o.d[r].z, g[j]);
                        m[in * V + j] = e * o.d[r].y;
                        m[in * V + NS + j] = o.d[r].z * hs[k][j];
                        w[k] = __builtin_fmaf(e, o.b[r][j], w[k]);
                        g[j] = e * (kKeep ? as[kKeep ? k : 0][j] : exp2_hw(o.d[r].x * A[j]));
                        const float q = g[j] * (k ? hs[k ? k - 1 : 0][j] : first[j]);
                        u[k] = __builtin_fmaf(A[j], q, u[k]);
                        da[j] = __builtin_fmaf(o.d[r].x, q, da[j]);
                    }
#pragma unroll
                    for (int j = 2 * NS; j < V; ++j) m[in * V + j] = 0.f;
                    if (in == 0) {
                        merge_all<CH / 2, 1, K>(m);
#pragma unroll
                        for (int q = 0; q < KEPT; ++q) {
                            const int at_v = mine + q * CH, row = k + at_v / V, val = at_v % V;
                            if (at_v < K && val < 2 * NS)
                                part[row * 2 * NP + (val < NS ? l.n0 + val : NP + l.n0 + val - NS)] = m[q];
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                merge_all<32, CH, GR>(w + i * GR);
                merge_all<32, CH, GR>(u + i * GR);
                ddelta[i] = (u[i * GR] * kLn2 + w[i * GR] * xf[i]) * sig[i];
                dx[i] = __builtin_fmaf(w[i * GR], d[i], skip * dv[i]);
                if (i * GR + l.row < rows) {
                    dskip = __builtin_fmaf(dv[i], xf[i], dskip);
                    dbias += ddelta[i];
                }
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) dA[j] += da[j];
            wx.template store<false>(a.dx ? rows : 0, dx);
            wd.template store<false>(a.ddelta ? rows : 0, ddelta);
            wz.template store<false>(a.dz ? rows : 0, dz);
            // The workgroup's sum of dB and dC; the other half of the buffer
            // is the next tile's, so one barrier a tile is enough.
            lds_barrier();
            float* out = a.part_bc + (static_cast<int64_t>(block) * a.part_rows + to) * 2 * a.n;
#pragma unroll
            for (int q = 0; q < (kTile * 2 * NP + kThreads - 1) / kThreads; ++q) {
                const int e = threadIdx.x + q * kThreads, row = e / (2 * NP), in = e % (2 * NP), n = in % NP;
                if (row < rows && n < a.n) {
                    const float* p = &lds_part[turn][0][e];
                    out[(row * 2 + in / NP) * a.n + n] = (p[0] + p[kTile * 2 * NP]) + (p[2 * kTile * 2 * NP] + p[3 * kTile * 2 * NP]);
                }
            }
            turn ^= 1;
        }
        if (a.dinitial && span.begin >= share.begin) l.write(a, a.dinitial + s * states, g);
    }
#pragma unroll
    for (int dist = 32; dist >= CH; dist >>= 1) {
        dskip += __shfl_xor(dskip, dist);
        dbias += __shfl_xor(dbias, dist);
    }
    float* part_a = a.part_a + item * states;
    const int64_t at_c = static_cast<int64_t>(item) * a.channels + l.c;
    if (a.seq0 > 0) {  // what the launch before has left there
        float before[NS];
        l.read(a, part_a, before);
#pragma unroll
        for (int j = 0; j < NS; ++j) dA[j] += before[j];
        dskip += a.part_d[at_c];
        dbias += a.part_bias[at_c];
    }
    l.write(a, part_a, dA);
    if (l.grp == 0 && l.on) {
        a.part_d[at_c] = dskip;
        a.part_bias[at_c] = dbias;
    }
    if (a.clear && a.starts) {  // rows of no sequence
        auto clear = [&](int64_t from, int64_t to) {
            if (a.dx) clear_rows<T>(l, a.dx, a.channels, from, to);
            if (a.ddelta) clear_rows<T>(l, a.ddelta, a.channels, from, to);
            if (a.dz) clear_rows<T>(l, a.dz, a.channels, from, to);
        };
        if (item == 0) clear(0, span_of(a, 0).begin);
        if (share.end_of_all) clear(span_of(a, a.seqs - 1).end, a.rows);
    }
}

// dB and dC: the sums over the workgroups of a group's channels, in order.
template <typename T>
__global__ __launch_bounds__(256) void sum_bc_kernel(ScanArgs a)
{
    const int64_t one = a.part_rows * 2 * a.n, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int group = blockIdx.y;
    if (at >= a.sum_rows * 2 * a.n) return;
    const int64_t in_launch = at / (2 * a.n), row = a.row0 + in_launch;
    const int in = static_cast<int>(at - in_launch * 2 * a.n), n = in % a.n;
    void* to = in < a.n ? a.dB : a.dC;
    if (!to) return;
    bool there = true;
    if (a.starts) there = row >= span_of(a, 0).begin && row < span_of(a, a.seqs - 1).end;
    float v = 0.f;
    if (there) {
        const float* p = a.part_bc + static_cast<int64_t>(group) * a.blocks * one + at;
        constexpr int kBatch = 8;
        for (int b = 0; b < a.blocks; b += kBatch) {
            float t[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) t[i] = b + i < a.blocks ? p[(b + i) * one] : 0.f;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v += t[i];
        }
    } else if (!a.clear) {
        return;
    }
    store_f(static_cast<T*>(to) + (row * a.groups + group) * a.n + n, v);
}

}  // namespace scan
}  // namespace convmi
