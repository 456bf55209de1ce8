// Forward pass of the selective scan, for one type: included by the sources
// that build it for bf16 and for fp32.
//
// What a state of a row costs are its instructions: d A, exp2 (a quarter of the
// rate), d x B, and the two multiply-adds of h and y are 8 issue slots; the
// rows' softplus, gate and conversions add about a third at 16 states.  Memory
// (x, delta, z, y once) takes a third of that time.
#pragma once

#include "scan.hpp"

namespace convmi {
namespace scan {

// The state that the pieces before a share leave to its first sequence: what
// each of them ends with, faded by the pieces between.
template <int GR, int NS>
__device__ __forceinline__ void inherit(const ScanArgs& a, const Lanes<GR, NS>& l, const float* A, int item, int64_t begin, float* h)
{
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    float passed = 0.f;
    for (int q = item - 1; q >= 0; --q) {
        float e[NS];
        l.read(a, a.ends + q * states, e);
        const float sum = a.sums[static_cast<int64_t>(q) * a.channels + l.c];
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = __builtin_fmaf(exp2_hw(A[j] * passed), e[j], h[j]);
        passed += sum;
        if (begin >= q * a.piece_rows) break;  // the sequence begins in that piece
    }
}

// kStates: states for the gradient's tiles alone; kEnds: the state at the end of
// a piece from nothing before it, for the pieces behind it.
enum Want { kOutputs, kStates, kEnds };

template <typename T, int GR, int NS, int WANT>
__global__ __launch_bounds__(kThreads) void fwd_kernel(ScanArgs a)
{
    typedef Lanes<GR, NS> L;
    constexpr int CH = L::CH, R = L::R, NP = L::NP;
    __shared__ float2 lds_d[kWaves][kTile][CH];
    __shared__ float lds_b[kWaves][kTile * NP], lds_c[kWaves][kTile * NP];

    const uint32_t cb = static_cast<uint32_t>(a.groups) * a.blocks;
    const int item = static_cast<int>(blockIdx.x / cb);
    const L l(a, blockIdx.x % cb);
    const Share share(a, item);
    float2(*dd)[CH] = lds_d[l.wave];
    float *sb = lds_b[l.wave], *sc = lds_c[l.wave];

    float A[NS], h[NS];
    l.read(a, a.A, A);
#pragma unroll
    for (int j = 0; j < NS; ++j) A[j] *= kLog2e;
    const float bias = a.bias ? a.bias[l.c] : 0.f, skip = a.D ? a.D[l.c] : 0.f;
    const int64_t states = static_cast<int64_t>(a.channels) * a.n;
    const bool gate = WANT == kOutputs && a.z;

    for (int s = share.first; s < share.last; ++s) {
        const Span span = span_of(a, s);
        if (WANT == kEnds && span.end <= share.end) continue;  // nothing goes on behind the piece
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = 0.f;
        if (span.begin >= share.begin) {
            if (a.initial) l.read(a, a.initial + s * states, h);
        } else if (WANT != kEnds) {
            inherit(a, l, A, item, span.begin, h);
        }
        int64_t at = span.begin > share.begin ? span.begin : share.begin;
        const int64_t end = span.end < share.end ? span.end : share.end;
        float total = 0.f;  // sum of d
        T x[R], dl[R], z[R];
        Shared<T, GR, NS> bc;
        auto fetch = [&](int64_t row0) __attribute__((always_inline)) {
            const int rows = static_cast<int>(tile_end(row0, end) - row0);
            load_rows(l, a.x, a.xs, row0, rows, x);
            load_rows(l, a.delta, a.ds, row0, rows, dl);
            if (gate) load_rows(l, a.z, a.zs, row0, rows, z);
            bc.load(a, l, row0, rows);
        };
        if (at < end) fetch(at);
        while (at < end) {
            const int64_t row0 = at;
            at = tile_end(at, end);
            const int rows = static_cast<int>(at - row0);
            float xf[R], zf[R], y[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = i * GR + l.row;
                xf[i] = load_f(&x[i]);
                zf[i] = gate ? load_f(&z[i]) : 0.f;
                float d = load_f(&dl[i]) + bias;
                if (a.softplus) d = softplus<false>(d).v;
                if (r >= rows) d = 0.f;  // a row that is not there changes nothing
                dd[r][l.ch] = make_float2(d, d * xf[i]);
            }
            bc.put(l, sb, sc);
            wave_fence();
            if (WANT != kEnds && a.saved && row0 > span.begin && (row0 & (kTile - 1)) == 0) l.write(a, a.saved + row0 / kTile * states, h);
            if (at < end) fetch(at);  // the next tile's loads run beside this tile's work
#pragma unroll
            for (int i = 0; i < R; ++i) {
                y[i] = 0.f;
                if (i * GR < rows) {
                    float v[GR];
#pragma unroll
                    for (int r = 0; r < GR; ++r) {
                        const float2 d = dd[i * GR + r][l.ch];
                        const float *b = sb + (i * GR + r) * NP + l.n0, *c = sc + (i * GR + r) * NP + l.n0;
                        if (WANT == kEnds) total += d.x;
                        v[r] = 0.f;
#pragma unroll
                        for (int j = 0; j < NS; ++j) {
                            h[j] = __builtin_fmaf(exp2_hw(d.x * A[j]), h[j], d.y * b[j]);
                            if (WANT == kOutputs) v[r] = __builtin_fmaf(h[j], c[j], v[r]);
                        }
                    }
                    if constexpr (WANT == kOutputs) {
                        merge_all<32, CH, GR>(v);
                        y[i] = __builtin_fmaf(skip, xf[i], v[0]);
                    }
                }
            }
            wave_fence();
            if constexpr (WANT == kOutputs) {
                if (gate)
                    with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                        for (int i = 0; i < R; ++i) y[i] *= act_value<kind()>(zf[i]);
                    });
                store_rows<T>(l, a.y, a.channels, row0, rows, y);
            }
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
