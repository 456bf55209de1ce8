// Gated feed-forward layer in bf16 on the matrix units:
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u,
//   dg = dh u act'(g),  du = dh act(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
//
// One product kernel serves all of it.  An output tile is BM "p" rows by BN
// "q" columns; the q operand is the matrix instruction's first (its rows are
// the output's contiguous dimension, so a lane ends with runs of four
// consecutive values of one output row):
//   forward, and g and u again:  p: rows of x,        q: rows of Wg and Wu
//   dx:                          p: rows of [dg|du],  q: columns of [Wg; Wu]
//   dW:                          p: columns of [dg|du], q: columns of x
// A wave's q tiles alternate between Wg and Wu in the forward product, so a
// lane holds g and u of the same elements and the activation, the product and
// the biases happen in registers.  Operands whose contraction index is
// contiguous are staged in LDS as rows of BK values, the others as they lie in
// memory, rows of one contraction index, and are read with the LDS transpose
// read.
//
// dg and du are rounded to bf16 once, as operands of the products that follow
// (their column sums, the bias gradients, are taken before); sums are fp32.
#include "gated.hpp"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace convmi {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;

enum Mode { kFwd, kAgain, kDx, kDw };

// WP x WQ waves, each TP x TQ tiles of 32x32; BK contraction values a stage.
template <int WP_, int WQ_, int TP_, int TQ_, int BK_, int NS_>
struct Shape {
    static constexpr int WP = WP_, WQ = WQ_, TP = TP_, TQ = TQ_, BK = BK_, NS = NS_;
    static constexpr int BM = WP * TP * 32, BN = WQ * TQ * 32, kThreads = WP * WQ * 64;
    static constexpr int kPBytes = BM * BK * 2, kQBytes = BN * BK * 2, kStage = kPBytes + kQBytes;
    static constexpr int kLds = NS * kStage;
    static constexpr int kPLoads = BM * BK / 8 / kThreads, kQLoads = BN * BK / 8 / kThreads;
    static constexpr int kLoads = kPLoads + kQLoads;
    static_assert(BM * BN * 2 <= kLds, "an output tile fits in the ring");
};

struct Product {
    const bf16_t *x, *wg, *wu, *bg, *bu, *dh;
    const bf16_t* d;      // [dg|du], rows of 2 Fp
    bf16_t *h, *out, *out2;  // out: dx, or dWg with dWu in out2
    bf16_t* d_out;
    float *saved, *sums, *part;
    int64_t rows, per;    // per: rows of a piece (dW)
    int C, F, Fp, act;
    int p_tiles, q_tiles;
};

// Where a 16-byte unit of a staged row sits.  Rows of BK values: 8 (or, with
// BK 32, 16) rows read at one unit reach all banks.  Rows of a contraction
// index: the four rows and four units of a transpose read do.
template <int BK>
__device__ __forceinline__ int swz_row(int r) { return BK == 64 ? (r & 7) : ((r >> 2) & 3); }
__device__ __forceinline__ int swz_k(int k) { return ((k & 3) << 2) ^ (k & 2); }

__device__ __forceinline__ uint4 guarded16(const bf16_t* p, int n)
{
    if (n >= 8) return load16_any(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) w[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stages R rows of K-contiguous data: units of row r from base + r * ld.  Two
// sources alternate every 32 rows when GATED.
template <typename S, int R, bool GATED, bool FAST>
struct RowStage {
    static constexpr int kUnits = S::BK / 8, kN = R * kUnits / S::kThreads;
    const bf16_t *src0, *src1;
    int valid;            // rows of a source
    int ld, K;
    __device__ __forceinline__ void issue(int kt, char* lds, int i) const
    {
        const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int idx = i * S::kThreads + tid;
        const int r = idx / kUnits, unit = (idx % kUnits) ^ swz_row<S::BK>(r);
        const int k = kt * S::BK + unit * 8;
        const int first = (i * S::kThreads + wave * 64) / kUnits;  // the wave's first row: one source a wave
        const int which = GATED ? (first >> 5) & 1 : 0;
        const int row = GATED ? (r >> 6) * 32 + (r & 31) : r;
        const bf16_t* src = GATED && which ? src1 : src0;
        if constexpr (FAST) {
            const uint32_t bytes = (static_cast<uint32_t>(valid) * ld - kt * S::BK) * 2;
            const uint32x4_t rs = dma_rsrc(src + kt * S::BK, valid > 0 ? bytes : 0u);
            const uint32_t off = (static_cast<uint32_t>(row) * ld + unit * 8) * 2;
            dma16(rs, k < K && row < valid ? off : kOutside, lds_addr(lds + (i * S::kThreads + wave * 64) * 16));
        } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < valid && k < K) v = guarded16(src + static_cast<int64_t>(row) * ld + k, K - k);
            *reinterpret_cast<uint4*>(lds + idx * 16) = v;
        }
    }
};

// Stages BK rows of a contraction index, R columns from `src`; `cols` of them
// exist, and `valid(kt)` rows.
template <typename S, int R, bool FAST>
struct ColStage {
    static constexpr int kUnits = R / 8, kN = R * S::BK / 8 / S::kThreads;
    __device__ __forceinline__ static void issue(const bf16_t* src, int valid, int ld, int cols, char* lds, int i)
    {
        const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int idx = i * S::kThreads + tid;
        const int k = idx / kUnits, unit = (idx % kUnits) ^ swz_k(k);
        if constexpr (FAST) {
            const uint32x4_t rs = dma_rsrc(src, valid > 0 ? (static_cast<uint32_t>(valid - 1) * ld + cols) * 2u : 0u);
            const uint32_t off = (static_cast<uint32_t>(k) * ld + unit * 8) * 2;
            dma16(rs, k < valid && unit * 8 < cols ? off : kOutside, lds_addr(lds + (i * S::kThreads + wave * 64) * 16));
        } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k < valid && unit * 8 < cols) v = guarded16(src + static_cast<int64_t>(k) * ld + unit * 8, cols - unit * 8);
            *reinterpret_cast<uint4*>(lds + idx * 16) = v;
        }
    }
};

// Reads fragments (8 contraction values of one row or column a lane) of tile
// `t` at step kk (16 values).
template <typename S>
struct RowFrag {
    int col, off[S::BK / 16];
    __device__ __forceinline__ RowFrag(int)
    {
        const int lane = threadIdx.x & 63;
        col = lane & 31;
#pragma unroll
        for (int kk = 0; kk < S::BK / 16; ++kk)
            off[kk] = col * (S::BK * 2) + (((kk * 2 + (lane >> 5)) ^ swz_row<S::BK>(col)) << 4);
    }
    __device__ __forceinline__ bf16x8 read(const lds_char* base, int tile, int, int kk) const
    {
        return *reinterpret_cast<const lds_bf16x8*>(base + tile * (32 * S::BK * 2) + off[kk]);
    }
};
template <typename S, int R, int T>
struct ColFrag {
    int off[T];
    __device__ __forceinline__ ColFrag(int tile0)
    {
        const int lane = threadIdx.x & 63, g4 = lane >> 4, s16 = lane & 15;
        const int k = 8 * (g4 >> 1) + (s16 >> 2);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int c = (tile0 + t) * 32 + 16 * (g4 & 1) + 4 * (s16 & 3);
            off[t] = k * (R * 2) + (((c >> 3) ^ swz_k(k)) << 4) + (c & 7) * 2;
        }
    }
    __device__ __forceinline__ bf16x8 read(const lds_char* base, int, int t, int kk) const
    {
        const lds_char* p = base + kk * 16 * (R * 2) + off[t];
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p);
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 4 * (R * 2)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// Writes a bf16 tile of `U` units a row from LDS to memory, whole units where
// they fit.  `row(r)` gives the address of row r, or null.
template <int U, int kThreads, typename F>
__device__ __forceinline__ void store_tile(const char* lds, int rows, int cols, F row)
{
    for (int idx = threadIdx.x; idx < rows * U; idx += kThreads) {
        const int r = idx / U, unit = (idx % U) ^ (r & 7);
        bf16_t* p = row(r);
        const int n = cols - unit * 8;
        if (!p || n <= 0) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + idx * 16);
        p += unit * 8;
        if (n >= 8) {
            store16_any(p, v);
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = static_cast<bf16_t>(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}
template <int U>
__device__ __forceinline__ int tile_byte(int r, int unit, int half) { return (r * U + (unit ^ (r & 7))) * 16 + half * 8; }

__device__ __forceinline__ void bias4(const bf16_t* b, int f, int F, float* v)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = b && f + e < F ? bf16_to_f(b[f + e]) : 0.f;
}

// Sums 16 values over the 32 lanes of a half wave; lane l of a half ends with
// value (l & 15)'s sum (in bit-reversed halves: see `which`).
__device__ __forceinline__ float half_sum16(float (&v)[16], int lane, int& which)
{
    which = 0;
#pragma unroll
    for (int s = 16, n = 8; n >= 1; s >>= 1, n >>= 1) {
        const bool up = lane & s;
        which += up ? n : 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor(send, s);
        }
    }
    return v[0] + __shfl_xor(v[0], 1);
}

// Tile of a workgroup.  Workgroup b runs on XCD b mod 8: each XCD takes a
// contiguous run of tiles, ordered so that eight p tiles share their q tiles.
__device__ __forceinline__ void pick_tile(int b, int n, int p_tiles, int q_tiles, int& pt, int& qt, int& piece)
{
    const int xcd = b & 7, per = n >> 3, rem = n & 7;
    int t = xcd * per + min(xcd, rem) + (b >> 3);
    const int tiles = p_tiles * q_tiles;
    piece = t / tiles;
    t -= piece * tiles;
    constexpr int kGroup = 8;
    const int g = t / (kGroup * q_tiles), in = t - g * kGroup * q_tiles;
    const int size = min(kGroup, p_tiles - g * kGroup);
    qt = in / size;
    pt = g * kGroup + in - qt * size;
}

template <typename S, int MODE, bool FAST>
__global__ __launch_bounds__(S::kThreads) void gated_product_kernel(Product a)
{
    extern __shared__ char ring[];
    constexpr bool kGated = MODE == kFwd || MODE == kAgain;
    constexpr bool kPRows = MODE != kDw, kQRows = kGated;
    constexpr int kQTile = kGated ? S::BN / 2 : S::BN;  // output columns of a tile
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave / S::WQ, wq = wave % S::WQ;
    const int col = lane & 31, q = lane >> 5;
    int pt, qt, piece;
    pick_tile(blockIdx.x, gridDim.x, a.p_tiles, a.q_tiles, pt, qt, piece);
    const int64_t p0 = static_cast<int64_t>(pt) * S::BM;
    const int q0 = qt * kQTile;

    // The contraction: K values from k0 on.
    const int64_t m0 = MODE == kDw ? piece * a.per : 0;
    const int64_t K = kGated ? a.C : MODE == kDx ? 2 * static_cast<int64_t>(a.Fp) : min(a.per, a.rows - m0);
    const int nk = static_cast<int>((K + S::BK - 1) / S::BK);
    const int rows_left = MODE == kDw ? 0 : static_cast<int>(min(static_cast<int64_t>(S::BM), a.rows - p0));

    auto issue = [&](int kt, char* st, int i) __attribute__((always_inline)) {
        if (i < S::kPLoads) {
            if constexpr (kPRows) {
                const int ld = kGated ? a.C : 2 * a.Fp;
                RowStage<S, S::BM, false, FAST> rs{(kGated ? a.x : a.d) + p0 * ld, nullptr, rows_left, ld, static_cast<int>(K)};
                rs.issue(kt, st, i);
            } else {
                const int64_t k = static_cast<int64_t>(kt) * S::BK;
                ColStage<S, S::BM, FAST>::issue(a.d + (m0 + k) * 2 * a.Fp + p0, static_cast<int>(min(K - k, static_cast<int64_t>(S::BK))),
                                                2 * a.Fp, static_cast<int>(2 * a.Fp - p0), st, i);
            }
        } else {
            char* qs = st + S::kPBytes;
            i -= S::kPLoads;
            if constexpr (kQRows) {
                const int64_t at = static_cast<int64_t>(q0) * a.C;
                RowStage<S, S::BN, true, FAST> rs{a.wg + at, a.wu + at, min(kQTile, a.F - q0), a.C, a.C};
                rs.issue(kt, qs, i);
            } else if constexpr (MODE == kDx) {
                const int k = kt * S::BK, up = k >= a.Fp, f = k - (up ? a.Fp : 0);
                ColStage<S, S::BN, FAST>::issue((up ? a.wu : a.wg) + static_cast<int64_t>(f) * a.C + q0, min(a.F - f, S::BK), a.C, a.C - q0, qs, i);
            } else {
                const int64_t k = static_cast<int64_t>(kt) * S::BK;
                ColStage<S, S::BN, FAST>::issue(a.x + (m0 + k) * a.C + q0, static_cast<int>(min(K - k, static_cast<int64_t>(S::BK))), a.C, a.C - q0, qs, i);
            }
        }
    };

    f32x16 acc[S::TQ][S::TP];
#pragma unroll
    for (int i = 0; i < S::TQ; ++i)
#pragma unroll
        for (int j = 0; j < S::TP; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

    typename std::conditional<kPRows, RowFrag<S>, ColFrag<S, S::BM, S::TP>>::type pf(wp * S::TP);
    typename std::conditional<kQRows, RowFrag<S>, ColFrag<S, S::BN, S::TQ>>::type qf(wq * S::TQ);
    struct Frags {
        bf16x8 q[S::TQ], p[S::TP];
    };
    auto read = [&](Frags& f, const char* st, int kk) __attribute__((always_inline)) {
        const lds_char* ps = (const lds_char*)st;
        const lds_char* qs = ps + S::kPBytes;
#pragma unroll
        for (int i = 0; i < S::TQ; ++i) f.q[i] = qf.read(qs, wq * S::TQ + i, i, kk);
#pragma unroll
        for (int j = 0; j < S::TP; ++j) f.p[j] = pf.read(ps, wp * S::TP + j, j, kk);
    };
    constexpr int kSteps = S::BK / 16;
    // Multiplies one stage; the loads of stage `next` go out between its steps.
    auto compute = [&](const char* st, int next, char* nst) __attribute__((always_inline)) {
        Frags f[2];
        read(f[0], st, 0);
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
            if (kk + 1 < kSteps) read(f[(kk + 1) & 1], st, kk + 1);
            if (next < nk) {
#pragma unroll
                for (int i = kk * S::kLoads / kSteps; i < (kk + 1) * S::kLoads / kSteps; ++i) issue(next, nst, i);
            }
#pragma unroll
            for (int i = 0; i < S::TQ; ++i)
#pragma unroll
                for (int j = 0; j < S::TP; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[kk & 1].q[i], f[kk & 1].p[j], acc[i][j], 0, 0, 0);
        }
    };

    // Stage kt has landed for every wave after its own wait and the barrier;
    // every wave is then done with stage kt - 1, whose place is filled next.
#pragma unroll
    for (int st = 0; st < S::NS - 1; ++st)
        if (st < nk)
            for (int i = 0; i < S::kLoads; ++i) issue(st, ring + st * S::kStage, i);
    for (int kt = 0; kt < nk; kt += S::NS) {
#pragma unroll
        for (int i = 0; i < S::NS; ++i)
            if (kt + i < nk) {
                if constexpr (FAST) {
                    if (kt + i + S::NS - 2 < nk) wait_vm_lds<(S::NS - 2) * S::kLoads>();
                    else wait_vm_lds<0>();
                    barrier_no_fence();
                } else {
                    __syncthreads();
                }
                compute(ring + i * S::kStage, kt + i + S::NS - 1, ring + (i + S::NS - 1) % S::NS * S::kStage);
            }
    }
    __syncthreads();  // every wave is done with the ring

    // A lane holds columns 8v + 4q + {0..3} of a q tile and p row `col`.
    if constexpr (kGated) {
        constexpr int U = kQTile / 8;  // units of a tile row
        char* second = ring + S::BM * kQTile * 2;
        if constexpr (MODE == kAgain) {
            // dh's tile, in the places that dg will take
            for (int idx = tid; idx < S::BM * U; idx += S::kThreads) {
                const int r = idx / U, f = q0 + ((idx % U) ^ (r & 7)) * 8;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows_left && f < a.F) v = guarded16(a.dh + (p0 + r) * a.F + f, a.F - f);
                *reinterpret_cast<uint4*>(ring + idx * 16) = v;
            }
            __syncthreads();
        }
        with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < S::TQ / 2; ++m) {
            const int base = (wq * (S::TQ / 2) + m) * 32;
            float sg[16], su[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) sg[v] = su[v] = 0.f;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int f = q0 + base + 8 * v + 4 * q;
                float bg[4], bu[4];
                bias4(a.bg, f, a.F, bg);
                bias4(a.bu, f, a.F, bu);
#pragma unroll
                for (int j = 0; j < S::TP; ++j) {
                    const int r = (wp * S::TP + j) * 32 + col;
                    char* at = ring + tile_byte<U>(r, base / 8 + v, q);
                    float g[4], u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[e] = acc[2 * m][j][4 * v + e] + bg[e];
                        u[e] = acc[2 * m + 1][j][4 * v + e] + bu[e];
                    }
                    if constexpr (MODE == kFwd) {
                        if (a.saved && r < rows_left) {
                            float* sp = a.saved + (p0 + r) * 2 * a.F + f;
                            if (f + 4 <= a.F) {
                                store16_any(sp, make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3])));
                                store16_any(sp + a.F, make_uint4(__float_as_uint(u[0]), __float_as_uint(u[1]), __float_as_uint(u[2]), __float_as_uint(u[3])));
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (f + e < a.F) sp[e] = g[e], sp[a.F + e] = u[e];
                            }
                        }
                        float h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = act_value<kind()>(g[e]) * u[e];
                        *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
                    } else {
                        const uint2 raw = *reinterpret_cast<const uint2*>(at);
                        const float dh[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                                             __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
                        float dg[4], du[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const ActPair p = act_pair<kind()>(g[e]);
                            dg[e] = dh[e] * u[e] * p.d;
                            du[e] = dh[e] * p.v;
                            sg[4 * v + e] += dg[e];
                            su[4 * v + e] += du[e];
                        }
                        *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3]));
                        *reinterpret_cast<uint2*>(at + S::BM * kQTile * 2) = make_uint2(pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3]));
                    }
                }
            }
            if constexpr (MODE == kAgain) {
                if (a.sums) {
                    int which;
                    const float tg = half_sum16(sg, lane, which), tu = half_sum16(su, lane, which);
                    const int f = q0 + base + 8 * (which >> 2) + 4 * q + (which & 3);
                    if ((lane & 1) == 0 && f < a.Fp) {
                        float* row = a.sums + static_cast<int64_t>(pt * S::WP + wp) * 2 * a.Fp;
                        row[f] = tg;
                        row[a.Fp + f] = tu;
                    }
                }
            }
        }
        });
        __syncthreads();
        if constexpr (MODE == kFwd) {
            store_tile<U, S::kThreads>(ring, S::BM, a.F - q0, [&](int r) { return r < rows_left ? a.h + (p0 + r) * a.F + q0 : nullptr; });
        } else {
            // the columns up to Fp too: their dh is 0, and so are they
            store_tile<U, S::kThreads>(ring, S::BM, a.Fp - q0, [&](int r) { return r < rows_left ? a.d_out + (p0 + r) * 2 * a.Fp + q0 : nullptr; });
            store_tile<U, S::kThreads>(second, S::BM, a.Fp - q0, [&](int r) { return r < rows_left ? a.d_out + (p0 + r) * 2 * a.Fp + a.Fp + q0 : nullptr; });
        }
    } else {
        // row p0 + r of the output: a row of dx, or of dWg or dWu (none: null)
        auto weight_row = [&](int64_t p, int64_t& f) {
            const bool up = p >= a.Fp;
            f = p - (up ? a.Fp : 0);
            return f < a.F && p < 2 * a.Fp ? (up ? 1 : 0) : -1;
        };
        if (MODE == kDw && a.part) {
#pragma unroll
            for (int j = 0; j < S::TP; ++j) {
                int64_t f;
                const int half = weight_row(p0 + (wp * S::TP + j) * 32 + col, f);
                if (half < 0) continue;
                float* row = a.part + ((static_cast<int64_t>(piece) * 2 + half) * a.F + f) * a.C;
#pragma unroll
                for (int i = 0; i < S::TQ; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int c = q0 + (wq * S::TQ + i) * 32 + 8 * v + 4 * q;
                        if (c + 4 <= a.C)
                            store16_any(row + c, make_uint4(__float_as_uint(acc[i][j][4 * v]), __float_as_uint(acc[i][j][4 * v + 1]),
                                                            __float_as_uint(acc[i][j][4 * v + 2]), __float_as_uint(acc[i][j][4 * v + 3])));
                        else
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (c + e < a.C) row[c + e] = acc[i][j][4 * v + e];
                    }
            }
            return;
        }
        constexpr int U = S::BN / 8;
#pragma unroll
        for (int i = 0; i < S::TQ; ++i)
#pragma unroll
            for (int j = 0; j < S::TP; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<uint2*>(ring + tile_byte<U>((wp * S::TP + j) * 32 + col, (wq * S::TQ + i) * 4 + v, q)) =
                        make_uint2(pack_bf16x2(acc[i][j][4 * v], acc[i][j][4 * v + 1]), pack_bf16x2(acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]));
        __syncthreads();
        store_tile<U, S::kThreads>(ring, S::BM, a.C - q0, [&](int r) -> bf16_t* {
            if (MODE == kDx) return r < rows_left && a.out ? a.out + (p0 + r) * a.C + q0 : nullptr;
            int64_t f;
            const int half = weight_row(p0 + r, f);
            bf16_t* w = half < 0 ? nullptr : half ? a.out2 : a.out;
            return w ? w + f * a.C + q0 : nullptr;
        });
    }
}

// Few rows: the layer is a stream over its weights.  A workgroup takes 16
// hidden channels (16 rows of Wg and of Wu), its waves share the contraction
// in pieces of 64 values, NP groups of 16 rows of x ride along, and the waves'
// sums are added in order.
constexpr int kFewWaves = 8;
template <int NP, bool FAST>
__global__ __launch_bounds__(kFewWaves * 64) void gated_few_rows_kernel(Product a)
{
    __shared__ f32x4 sums[kFewWaves][2][NP][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 15, ku = (lane >> 4) * 8;
    const int f0 = blockIdx.x * 16;
    const int64_t fr = min(f0 + row, a.F - 1);
    const bf16_t *wg = a.wg + fr * a.C, *wu = a.wu + fr * a.C;
    const bf16_t* x[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) x[j] = a.x + min(static_cast<int64_t>(j * 16 + row), a.rows - 1) * a.C;
    f32x4 g[NP], u[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) g[j] = u[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto load = [&](const bf16_t* p, int k) __attribute__((always_inline)) {
        if (k >= a.C) return make_uint4(0, 0, 0, 0);
        return FAST ? *reinterpret_cast<const uint4*>(p + k) : guarded16(p + k, a.C - k);
    };
    constexpr int U = NP == 1 ? 2 : 1;  // pieces in flight
    for (int k0 = wave * 64; k0 < a.C; k0 += kFewWaves * 64 * U) {
        uint4 vg[U][2], vu[U][2], vx[U][2][NP];
#pragma unroll
        for (int t = 0; t < U; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = k0 + t * kFewWaves * 64 + s * 32 + ku;
                vg[t][s] = load(wg, k);
                vu[t][s] = load(wu, k);
#pragma unroll
                for (int j = 0; j < NP; ++j) vx[t][s][j] = load(x[j], k);
            }
#pragma unroll
        for (int t = 0; t < U; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const bf16x8 b = __builtin_bit_cast(bf16x8, vx[t][s][j]);
                    g[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vg[t][s]), b, g[j], 0, 0, 0);
                    u[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vu[t][s]), b, u[j], 0, 0, 0);
                }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        sums[wave][0][j][lane] = g[j];
        sums[wave][1][j][lane] = u[j];
    }
    __syncthreads();
    // value (p, f): lane (f / 4) * 16 + p of a group, element f % 4
    for (int idx = threadIdx.x; idx < NP * 256; idx += kFewWaves * 64) {
        const int f = idx & 15, p = idx >> 4;
        if (p >= a.rows || f0 + f >= a.F) continue;
        const int at = (f >> 2) * 16 + (p & 15);
        float gv = 0.f, uv = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) {
            gv += reinterpret_cast<const float*>(&sums[w][0][p >> 4][at])[f & 3];
            uv += reinterpret_cast<const float*>(&sums[w][1][p >> 4][at])[f & 3];
        }
        if (a.bg) gv += bf16_to_f(a.bg[f0 + f]), uv += bf16_to_f(a.bu[f0 + f]);
        if (a.saved) {
            a.saved[static_cast<int64_t>(p) * 2 * a.F + f0 + f] = gv;
            a.saved[static_cast<int64_t>(p) * 2 * a.F + a.F + f0 + f] = uv;
        }
        a.h[static_cast<int64_t>(p) * a.F + f0 + f] = f_to_bf16(act_value(a.act, gv) * uv);
    }
}

typedef Shape<2, 4, 4, 2, 64, 2> Big;    // 256 x 256, eight waves
typedef Shape<2, 2, 2, 2, 64, 2> Small;  // 128 x 128, four waves

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int64_t tiles(int64_t n, int t) { return (n + t - 1) / t; }

template <typename S, int MODE, bool FAST>
hipError_t run(Product& k, int64_t p_tiles, int64_t q_tiles, int pieces, hipStream_t s)
{
    k.p_tiles = static_cast<int>(p_tiles);
    k.q_tiles = static_cast<int>(q_tiles);
    const int64_t blocks = p_tiles * q_tiles * pieces;
    if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    auto kernel = gated_product_kernel<S, MODE, FAST>;
    static std::atomic<bool> ready{false};
    if (S::kLds > 65536 && !ready.load(std::memory_order_acquire)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
        if (e != hipSuccess) return e;
        ready.store(true, std::memory_order_release);
    }
    return launch(kernel, dim3(static_cast<unsigned>(blocks)), dim3(S::kThreads), S::kLds, s, k);
}

// The large tile once it gives every CU one; smaller ones below that.
bool use_big(int64_t p, int64_t q, int pieces) { return tiles(p, Big::BM) * tiles(q, Big::BN) * pieces >= device_cu_count(); }

template <int MODE>
hipError_t run_tiles(Product& k, int64_t p, int64_t q, int pieces, bool big, bool fast, hipStream_t s)
{
    if (big) {
        const int64_t pt = tiles(p, Big::BM), qt = tiles(q, Big::BN);
        return fast ? run<Big, MODE, true>(k, pt, qt, pieces, s) : run<Big, MODE, false>(k, pt, qt, pieces, s);
    }
    const int64_t pt = tiles(p, Small::BM), qt = tiles(q, Small::BN);
    return fast ? run<Small, MODE, true>(k, pt, qt, pieces, s) : run<Small, MODE, false>(k, pt, qt, pieces, s);
}

Product product(const GatedArgs& a)
{
    Product k{};
    k.x = static_cast<const bf16_t*>(a.x);
    k.wg = static_cast<const bf16_t*>(a.wg);
    k.wu = static_cast<const bf16_t*>(a.wu);
    k.bg = static_cast<const bf16_t*>(a.bg);
    k.bu = static_cast<const bf16_t*>(a.bu);
    k.dh = static_cast<const bf16_t*>(a.dh);
    k.rows = a.rows;
    k.C = a.C;
    k.F = a.F;
    k.act = a.act;
    return k;
}

constexpr int64_t kFewRows = 64;

}  // namespace

GatedPlan gated_plan_bf16(int64_t rows, int C, int F)
{
    GatedPlan p{};
    p.Fp = (F + 63) / 64 * 64;
    // pieces of the weight gradients' sum: about one workgroup a CU, no piece
    // under 512 rows
    const bool big = use_big(2 * static_cast<int64_t>(p.Fp), C, 1);
    const int bm = big ? Big::BM : Small::BM, bn = big ? Big::BN : Small::BN;
    const int64_t t = tiles(2 * static_cast<int64_t>(p.Fp), bm) * tiles(C, bn);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>((big ? 1 : 2) * device_cu_count() / t, rows / 512));
    p.per = std::max<int64_t>(64, (tiles(rows, static_cast<int>(want)) + 63) / 64 * 64);
    p.pieces = static_cast<int>(std::max<int64_t>(1, (rows + p.per - 1) / p.per));
    int64_t chunk;
    const int64_t again = tiles(rows, Small::BM) * Small::WP;
    p.sum_rows = static_cast<int>(std::max<int64_t>(gated_kept_chunks(rows, p.Fp, &chunk), again));
    p.d_bytes = round256(static_cast<size_t>(rows) * 2 * p.Fp * 2);
    p.sum_bytes = round256(static_cast<size_t>(p.sum_rows) * 2 * p.Fp * 4);
    p.part_bytes = p.pieces > 1 ? round256(static_cast<size_t>(p.pieces) * 2 * F * C * 4) : 0;
    return p;
}

hipError_t gated_fwd_bf16(const GatedArgs& a, hipStream_t s)
{
    Product k = product(a);
    k.h = static_cast<bf16_t*>(a.h);
    k.saved = a.saved;
    const bool fast = a.C % 8 == 0 && aligned(a.x) && aligned(a.wg) && aligned(a.wu);
    if (a.rows <= kFewRows) {
        const dim3 grid((a.F + 15) / 16), block(kFewWaves * 64);
        if (a.rows <= 16) return launch(fast ? gated_few_rows_kernel<1, true> : gated_few_rows_kernel<1, false>, grid, block, 0, s, k);
        if (a.rows <= 32) return launch(fast ? gated_few_rows_kernel<2, true> : gated_few_rows_kernel<2, false>, grid, block, 0, s, k);
        return launch(fast ? gated_few_rows_kernel<4, true> : gated_few_rows_kernel<4, false>, grid, block, 0, s, k);
    }
    return run_tiles<kFwd>(k, a.rows, 2 * static_cast<int64_t>(a.F), 1, use_big(a.rows, 2 * static_cast<int64_t>(a.F), 1), fast, s);
}

hipError_t gated_bwd_bf16(const GatedArgs& a, hipStream_t s)
{
    const GatedPlan p = gated_plan_bf16(a.rows, a.C, a.F);
    char* ws = static_cast<char*>(a.workspace);
    bf16_t* d = reinterpret_cast<bf16_t*>(ws);
    float* sums = a.dbg || a.dbu ? reinterpret_cast<float*>(ws + p.d_bytes) : nullptr;
    float* part = reinterpret_cast<float*>(ws + p.d_bytes + p.sum_bytes);
    const ArmedEvents armed = armed_events();
    armed_events() = ArmedEvents{armed.start, nullptr};
    hipError_t e = hipSuccess;
    int sum_rows = 0;
    if (a.rows > 0) {
        if (a.saved) {
            int64_t chunk;
            sum_rows = gated_kept_chunks(a.rows, p.Fp, &chunk);
            e = launch_gated_kept(a, d, sums, p.Fp, sum_rows, chunk, 1, s);
        } else {
            Product k = product(a);
            k.d_out = d;
            k.sums = sums;
            k.Fp = p.Fp;
            const bool fast = a.C % 8 == 0 && aligned(a.x) && aligned(a.wg) && aligned(a.wu);
            const bool big = use_big(a.rows, 2 * static_cast<int64_t>(a.F), 1);
            sum_rows = static_cast<int>(tiles(a.rows, big ? Big::BM : Small::BM)) * (big ? Big::WP : Small::WP);
            e = run_tiles<kAgain>(k, a.rows, 2 * static_cast<int64_t>(a.F), 1, big, fast, s);
        }
        armed_events() = ArmedEvents{nullptr, nullptr};
        if (e != hipSuccess) return e;
        if (a.dx) {
            Product k = product(a);
            k.d = d;
            k.Fp = p.Fp;
            k.out = static_cast<bf16_t*>(a.dx);
            e = run_tiles<kDx>(k, a.rows, a.C, 1, use_big(a.rows, a.C, 1), a.C % 8 == 0 && aligned(a.wg) && aligned(a.wu), s);
            if (e != hipSuccess) return e;
        }
    }
    if (sums) {
        e = launch_gated_bias_sums(a, sums, sum_rows, p.Fp, 1, s);
        if (e != hipSuccess) return e;
    }
    if (a.dwg || a.dwu) {
        Product k = product(a);
        k.d = d;
        k.Fp = p.Fp;
        k.out = static_cast<bf16_t*>(a.dwg);
        k.out2 = static_cast<bf16_t*>(a.dwu);
        k.part = p.pieces > 1 ? part : nullptr;
        k.per = p.per;
        if (p.pieces == 1) armed_events() = ArmedEvents{nullptr, armed.stop};
        e = run_tiles<kDw>(k, 2 * static_cast<int64_t>(p.Fp), a.C, p.pieces, use_big(2 * static_cast<int64_t>(p.Fp), a.C, 1),
                           a.C % 8 == 0 && aligned(a.x), s);
        armed_events() = ArmedEvents{nullptr, p.pieces > 1 ? armed.stop : nullptr};
        if (e == hipSuccess && p.pieces > 1) e = launch_gated_weight_sums(a, part, p.pieces, 1, s);
    }
    armed_events() = ArmedEvents{nullptr, nullptr};
    return e;
}

}  // namespace convmi
