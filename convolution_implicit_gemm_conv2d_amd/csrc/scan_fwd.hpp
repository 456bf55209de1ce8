// Forward pass of the selective scan, for one type: included by the sources
// that build it for bf16 and for fp32.
//
// What a state of a row costs are its instructions: d A, exp2, d x B, and the two
// multiply-adds of h and y take 20 cycles of a SIMD with eight waves, 22.6 with two (exp2
// alone 8.6); the row's softplus, gate, conversions and merges come on top.  4 x 4096 rows
// of 4096 channels, 16 states, bf16: 370 to 382 us (fp32 402), where the states alone are
// 137 at eight waves and memory (x, delta, z, y once) 104.  A wave's tile of 16 rows is 268
// vector instructions, 40 of them exp2, that keep the vector units busy 87 % of the
// time; LDS is busy 61 % of it, and no line is fetched twice (412 MB read, 150 written).
// 16384 rows of 1024 channels in 32 pieces, 144 us: two fifths of it for their ends.
#pragma once

#include "scan.hpp"

namespace convmi {
namespace scan {

// kStates: states for the gradient's tiles alone; kEnds: the state at the end of
// a piece from nothing before it, for the pieces behind it.
enum Want { kOutputs, kStates, kEnds };
constexpr int kAhead = 2;

template <typename T, int GR, int NS, int WANT>
__global__ __launch_bounds__(kThreads) void fwd_kernel(ScanArgs a)
{
    typedef Lanes<GR, NS> L;
    constexpr int CH = L::CH, R = L::R, LP = L::LP;
    // two tiles: while one is worked on, the next one is prepared
    __shared__ float2 lds_d[kWaves][2][kTile][CH];
    __shared__ float lds_b[kWaves][2][kTile * LP], lds_c[kWaves][2][kTile * LP];

    const uint32_t cb = static_cast<uint32_t>(a.groups) * a.blocks;
    const int item = static_cast<int>(blockIdx.x / cb);
    const L l(a, blockIdx.x % cb);
    const Share share(a, item);

    float A[NS], h[NS];
    l.read(a, a.A, A);
#pragma unroll
    for (int j = 0; j < NS; ++j) A[j] *= kLog2e;
    const float bias = a.bias ? a.bias[l.c] : 0.f, skip = a.D ? a.D[l.c] : 0.f;
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    const bool gate = WANT == kOutputs && a.z;
    const States<GR, NS> kept(a, l);

    for (int s = share.first; s < share.last; ++s) {
        const Span span = span_of(a, s);
        if (WANT == kEnds && span.end <= share.end) continue;  // nothing goes on behind the piece
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = 0.f;
        if (span.begin >= share.begin) {
            if (a.initial) l.read(a, a.initial + s * states, h);
        } else if (WANT != kEnds) {
            inherit<-1>(a, l, A, item, item - piece_of(a, span.begin), h);
        }
        const int begin = span.begin > share.begin ? span.begin : share.begin, end = span.end < share.end ? span.end : share.end;
        float total = 0.f;  // sum of d
        Rows<T, GR, NS> rx(l, a.x, a.xs, begin), rd(l, a.delta, a.ds, begin), rz(l, a.z, a.zs, begin), ry(l, a.y, a.channels, begin);
        // Loads run kAhead tiles ahead of the work, each tile's in registers of
        // its own.
        struct Raw {
            T x[R], dl[R], z[R], b[L::LOADS], c[L::LOADS];
        };
        Shared<T, GR, NS> bc(a, l, begin);
        Raw raw[kAhead];
        // Without a condition: a wait for one tile's loads can then leave the
        // later ones in flight (past the end they are of no rows).
        int ahead = begin;
        auto load_next = [&](Raw& w) __attribute__((always_inline)) {
            const int n = rows_from(ahead, end);
            rx.template load<true>(n, w.x);
            rd.template load<true>(n, w.dl);
            rz.template load<true>(gate ? n : 0, w.z);
            bc.template load<true>(n, w.b, w.c);
            ahead += n;
        };
        // A tile's steps and inputs, from registers to LDS.
        struct Ready {
            float x[R], z[R], d[R];
        };
        auto prepare = [&](const Raw& w, int rows, Ready& v) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                v.x[i] = load_f(&w.x[i]);
                v.z[i] = load_f(&w.z[i]);
                const float t = load_f(&w.dl[i]) + bias, p = softplus<false>(t).v;
                v.d[i] = a.softplus ? p : t;
                if (i * GR + l.row >= rows) v.d[i] = 0.f;  // a row that is not there changes nothing
            }
        };
        auto put_tile = [&](const Raw& w, const Ready& v, int turn) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < R; ++i) lds_d[l.wave][turn][i * GR + l.row][l.ch] = make_float2(v.d[i], v.d[i] * v.x[i]);
            bc.put(w.b, w.c, lds_b[l.wave][turn], lds_c[l.wave][turn]);
        };
        typedef Operands<NS, kGroup, float2> Ops;
        Ops ops[2];
        auto fetch = [&](Ops& o, int turn, int row) __attribute__((always_inline)) {
#pragma unroll
            for (int r = 0; r < kGroup; ++r) {
                o.d[r] = lds_d[l.wave][turn][row + r][l.ch];
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    o.b[r][j] = lds_b[l.wave][turn][(row + r) * LP + l.grp * L::SP + j];
                    if (WANT == kOutputs) o.c[r][j] = lds_c[l.wave][turn][(row + r) * LP + l.grp * L::SP + j];
                }
            }
        };
        Ready now, next;
        int at = begin, rows = 0;
        if (begin < end) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load_next(raw[k]);
            rows = rows_from(at, end);
            prepare(raw[0], rows, now);
            wave_fence();
            put_tile(raw[0], now, 0);
            load_next(raw[0]);
            wave_fence();
            fetch(ops[0], 0, 0);
        }
        // One tile, which is in LDS, and beside it the next one's preparation:
        // dependent chains that cost little time of their own there.
        auto work = [&](Raw& w, int turn) __attribute__((always_inline)) {
            const int here = rows;
            if (WANT != kEnds && a.saved && at > span.begin)
                kept.put(make_rsrc(a.saved + static_cast<int64_t>(at / kTile) * states, static_cast<uint32_t>(states) * 4), h);
            at += rows;
            rows = rows_from(at, end);
            prepare(w, rows, next);
            float v[kTile], y[R];
#pragma unroll
            for (int g = 0; g < kTile / kGroup; ++g) {
                if (g + 1 < kTile / kGroup) {
                    fetch(ops[(g + 1) & 1], turn, (g + 1) * kGroup);
                } else {
                    wave_fence();
                    put_tile(w, next, turn ^ 1);
                    load_next(w);
                    wave_fence();
                    fetch(ops[0], turn ^ 1, 0);
                }
                lds_stays();
                const Ops& o = ops[g & 1];
#pragma unroll
                for (int r = 0; r < kGroup; ++r) {
                    if (WANT == kEnds) total += o.d[r].x;
                    float acc = 0.f;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        h[j] = __builtin_fmaf(exp2_hw(o.d[r].x * A[j]), h[j], o.d[r].y * o.b[r][j]);
                        if (WANT == kOutputs) acc = __builtin_fmaf(h[j], o.c[r][j], acc);
                    }
                    v[g * kGroup + r] = acc;
                }
            }
            if constexpr (WANT == kOutputs) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    merge_all<32, CH, GR>(v + i * GR);
                    y[i] = __builtin_fmaf(skip, now.x[i], v[i * GR]);
                }
                if (gate)
                    with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                        for (int i = 0; i < R; ++i) y[i] *= act_value<kind()>(now.z[i]);
                    });
                ry.template store<true>(here, y);
            }
            now = next;
        };
        static_assert(kAhead == 2 && kTile / kGroup % 2 == 0, "registers and LDS alternate");
        while (at < end) {
            work(raw[1], 0);
            if (at < end) work(raw[0], 1);
        }
        if (WANT == kOutputs && a.last && span.end <= share.end) l.write(a, a.last + s * states, h);
        if (WANT == kEnds) {
            l.write(a, a.ends + item * states, h);
            if (l.grp == 0 && l.on) a.sums[static_cast<int64_t>(item) * a.channels + l.c] = total;
        }
    }
    if (WANT == kOutputs && a.clear && a.starts) {  // rows of no sequence
        if (item == 0) clear_rows<T>(l, a.y, a.channels, 0, span_of(a, 0).begin);
        if (share.end_of_all) clear_rows<T>(l, a.y, a.channels, span_of(a, a.seqs - 1).end, a.rows);
    }
}

}  // namespace scan
}  // namespace convmi
