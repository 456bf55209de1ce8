// Gated feed-forward layer on the matrix units, for bf16 (T bf16_t) and fp32:
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
// lane holds g and u of the same elements and the activation and the product
// happen in registers; the biases are the accumulators' first values.
// Operands whose contraction index is contiguous are staged in LDS as rows of
// BK values, the others as they lie in memory, rows of one contraction index,
// and are read with the LDS transpose read (bf16) or value by value (fp32).
// A step of 32 bytes of contraction values a row is one 32x32x16 instruction
// in bf16, four 32x32x2 in fp32: of those, instruction e multiplies the values
// e of the two 16-byte units that the half waves hold of a row.
//
// What bounds it: matrix instructions, up to the card's power (long sums: 1160 to
// 1180 TFLOP/s on normal data at a clock near 2.0 GHz, 1820 on zeros), or for
// short sums the epilogue's vector instructions (100352 rows, 256 -> 2 x 1024:
// 175 us, 87 of them products), or for few rows the weights' stream (one row,
// 2048 -> 2 x 8192: 15.2 us, 4.4 TB/s, with weights that no cache holds; 11.8
// where the memory-side cache has them from the call before).
//
// dg and du are rounded to T once, as operands of the products that follow
// (their column sums, the bias gradients, are taken before); sums are fp32.
#pragma once

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

enum Mode { kFwd, kAgain, kDx, kDw };

// WP x WQ waves, each TP x TQ tiles of 32x32; BK contraction values a stage,
// NS stages in the ring.
template <typename T_, int WP_, int WQ_, int TP_, int TQ_, int BK_, int NS_>
struct Shape {
    typedef T_ T;
    static constexpr int E = sizeof(T), kUnit = 16 / E;  // values of a 16-byte unit
    static constexpr int WP = WP_, WQ = WQ_, TP = TP_, TQ = TQ_, BK = BK_, NS = NS_;
    static constexpr int BM = WP * TP * 32, BN = WQ * TQ * 32, kThreads = WP * WQ * 64;
    static constexpr int kRowBytes = BK * E, kSteps = kRowBytes / 32;
    static constexpr int kPBytes = BM * kRowBytes, kQBytes = BN * kRowBytes, kStage = kPBytes + kQBytes;
    static constexpr int kLds = NS * kStage + BN * 4;  // the ring and a tile's biases
    static constexpr int kPLoads = kPBytes / 16 / kThreads, kQLoads = kQBytes / 16 / kThreads;
    static constexpr int kLoads = kPLoads + kQLoads;
    static constexpr int kWaveLds = kStage / (WP * WQ);  // a wave's part of a stage
    // of a SIMD: the accumulators take 16 TP TQ of its 512 registers
    static constexpr int kWaves = TP * TQ > 8 ? 1 : TP * TQ > 2 ? 2 : 3;
    static constexpr int kPerCu = 163840 / kLds < 4 * kWaves / (WP * WQ) ? 163840 / kLds : 4 * kWaves / (WP * WQ);  // workgroups
    static_assert(kPerCu > 0 && BN <= kThreads, "");
    static_assert(kWaveLds >= 4096, "a wave's output passes through its part of a stage");
    static_assert(kPLoads > 0 && kQLoads > 0 && TQ % 2 == 0 && NS >= 2, "");
    static_assert((kRowBytes == 64 || kRowBytes == 128) && 64 % BK == 0, "");
};

template <typename T>
struct Product {
    const T *x, *wg, *wu, *bg, *bu, *dh;
    const T* d;           // [dg|du], rows of 2 Fp
    T *h, *out, *out2;    // out: dx, or dWg with dWu in out2
    T* d_out;
    float *saved, *sums, *part;
    int64_t rows, per;    // per: contraction values of a piece (dx, dW)
    int C, F, Fp, act;
    int x_ld, w_ld;       // row pitches of x and of the weights: C, or that of their padded copies
    int p_tiles, q_tiles, tiles;  // tiles: of all pieces
};

// Where a 16-byte unit of a staged row sits.  Rows of contraction values: the
// 8 (rows of 128 bytes) or 16 (of 64) rows read at one unit reach all banks.
// Rows of a contraction index: the four rows and four units of a transpose
// read do (bf16), or the two rows that the half waves read (fp32).
template <int BYTES>
__device__ __forceinline__ int swz_row(int r) { return BYTES == 128 ? (r & 7) : ((r >> 2) & 3); }
template <typename T>
__device__ __forceinline__ int swz_k(int k) { return sizeof(T) == 2 ? ((k & 3) << 2) ^ (k & 2) : (k & 4) << 1; }

// A unit's worth of values at byte `off` of a buffer at any element alignment,
// none where it is kOutside.  `ragged` (uniform: the last unit of some row is
// cut): the first n of them by elements.  No branches but the uniform one.
constexpr uint32_t kAll = 0x7ffffffcu;
template <typename T>
__device__ __forceinline__ uint4 unit_load(rsrc_t r, uint32_t off, bool ragged, int n)
{
    if (!ragged) return buffer_load16(r, off);
    uint32_t w[4] = {0, 0, 0, 0};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e >> 1] |= static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(r, e < n ? off + 2 * e : kOutside, 0, 0)) << (16 * (e & 1));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_raw_buffer_load_b32(r, e < n ? off + 4 * e : kOutside, 0, 0);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Addresses of one operand's units for a thread: `off` within a tile (kOutside
// where the tile's row or column does not exist) and the unit's contraction
// offset.  ROWS: R rows of contraction values; otherwise BK rows of a
// contraction index with R columns each.
template <typename S, int R, bool ROWS>
struct Units {
    static constexpr int kN = R * S::kRowBytes / 16 / S::kThreads, kRow = ROWS ? S::kRowBytes / 16 : R / S::kUnit;
    uint32_t off[kN];
    // contraction offset (within a stage) of unit i of this thread
    static __device__ __forceinline__ int k(int i)
    {
        const int idx = i * S::kThreads + threadIdx.x, r = idx / kRow;
        return ROWS ? ((idx % kRow) ^ swz_row<S::kRowBytes>(r)) * S::kUnit : r;
    }
    // `valid` rows (ROWS) or columns of the tile exist.  GATED: two sources
    // alternate every 32 rows.
    template <bool GATED>
    __device__ __forceinline__ void set(int valid, int ld)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int idx = i * S::kThreads + threadIdx.x, r = idx / kRow;
            if (ROWS) {
                const int row = GATED ? (r >> 6) * 32 + (r & 31) : r;
                off[i] = row < valid ? (static_cast<uint32_t>(row) * ld + k(i)) * S::E : kOutside;
            } else {
                const int c = ((idx % kRow) ^ swz_k<typename S::T>(r)) * S::kUnit;
                off[i] = c < valid ? (static_cast<uint32_t>(r) * ld + c) * S::E : kOutside;
            }
        }
    }
    // Drops the units past `left` contraction values.
    __device__ __forceinline__ void cut(int left)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) off[i] = k(i) < left ? off[i] : kOutside;
    }
    // GATED: whether unit i of this wave comes from the second source.
    static __device__ __forceinline__ int second(int i)
    {
        return (((i * S::kThreads + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64) / kRow) >> 5) & 1;
    }
    // Values of unit i that exist, for the guarded loads.
    __device__ __forceinline__ int count(int i, int k_left, int valid) const
    {
        if (off[i] == kOutside) return 0;
        if (ROWS) return k_left - k(i);
        const int idx = i * S::kThreads + threadIdx.x, r = idx / kRow;
        return r < k_left ? valid - ((idx % kRow) ^ swz_k<typename S::T>(r)) * S::kUnit : 0;
    }
};

// Reads fragments (16 bytes of contraction values of one row or column a lane)
// of tile `t` at step kk.
template <typename S>
struct RowFrag {
    int off[S::kSteps];
    __device__ __forceinline__ RowFrag(int)
    {
        const int lane = threadIdx.x & 63, col = lane & 31;
#pragma unroll
        for (int kk = 0; kk < S::kSteps; ++kk)
            off[kk] = col * S::kRowBytes + (((kk * 2 + (lane >> 5)) ^ swz_row<S::kRowBytes>(col)) << 4);
    }
    __device__ __forceinline__ f32x4 read(const lds_char* base, int tile, int, int kk) const
    {
        return *reinterpret_cast<const __attribute__((address_space(3))) f32x4*>(base + tile * (32 * S::kRowBytes) + off[kk]);
    }
};
template <typename S, int R, int T>
struct ColFrag {
    int off[T];
    __device__ __forceinline__ ColFrag(int tile0)
    {
        const int lane = threadIdx.x & 63, g4 = lane >> 4, s16 = lane & 15;
        const int k = S::E == 2 ? 8 * (g4 >> 1) + (s16 >> 2) : 4 * (lane >> 5);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int c = (tile0 + t) * 32 + (S::E == 2 ? 16 * (g4 & 1) + 4 * (s16 & 3) : lane & 31);
            off[t] = k * (R * S::E) + (((c / S::kUnit) ^ swz_k<typename S::T>(k)) << 4) + c % S::kUnit * S::E;
        }
    }
    __device__ __forceinline__ f32x4 read(const lds_char* base, int, int t, int kk) const
    {
        const lds_char* p = base + kk * (32 / S::E) * (R * S::E) + off[t];
        if constexpr (S::E == 2) {
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p);
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 4 * (R * 2)));
            return __builtin_bit_cast(f32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const __attribute__((address_space(3))) float*>(p + e * (R * 4));
            return v;
        }
    }
};
template <typename T>
__device__ __forceinline__ f32x16 multiply(f32x4 q, f32x4 p, f32x16 acc)
{
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(q[e], p[e], acc, 0, 0, 0);
        return acc;
    }
}

// A wave's 32 output rows on their way from the accumulators' layout (a lane
// holds columns 8v + 4q + {0..3} of row `lane & 31`) to rows in memory: through
// the wave's own part of LDS, U units of 16 bytes a row, so that a store
// instruction writes whole lines.  LDS serves a wave in order; only the
// compiler has to keep the order too.
__device__ __forceinline__ void wave_order()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}
template <int U>
__device__ __forceinline__ int turn_at(int r, int unit) { return (r * U + (unit ^ ((r >> (U == 8 ? 1 : 2)) & (U - 1)))) * 16; }

// `cols` columns of T exist from `p` (uniform) on, `rows` rows of pitch ld.
template <int U, typename T>
__device__ __forceinline__ void turn_out(const char* lds, T* p, uint32_t ld, int rows, int cols)
{
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const rsrc_t out = make_rsrc(p, kAll);
    const bool ragged = cols < U * V && cols % V != 0;
#pragma unroll
    for (int i = 0; i < U / 2; ++i) {
        const int r = (i * 64 + lane) / U, unit = lane % U, n = cols - unit * V;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + turn_at<U>(r, unit));
        const uint32_t off = r < rows && n > 0 ? (r * ld + unit * V) * static_cast<uint32_t>(sizeof(T)) : kOutside;
        if (!ragged) {
            buffer_store16(out, off, v);
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const uint32_t at = e < n && off != kOutside ? off + e * static_cast<uint32_t>(sizeof(T)) : kOutside;
                if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1))), out, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(w[e], out, at, 0, 0);
            }
        }
    }
}

// Sums 16 values over the 32 lanes of a half wave: in each step a lane gives
// half of its values to a partner and keeps the other half.  A lane ends with
// the sum of value half_sum_of(lane).
__device__ __forceinline__ int half_sum_of(int lane) { return lane >> 1 & 15; }
template <int CTRL, int N>
__device__ __forceinline__ void half_sum_step(float* v, bool up)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float send = up ? v[i] : v[i + N], keep = up ? v[i + N] : v[i];
        v[i] = keep + dpp_shift<CTRL, 0xf>(send);
    }
}
__device__ __forceinline__ float half_sum16(float (&v)[16], int lane)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // swaps the odd rows of 16 lanes of one with the even ones of the other
        const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 8]), false, false);
        v[i] = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    }
    half_sum_step<0x140, 4>(v, lane & 8);  // lane 15 - i of a row
    half_sum_step<0x141, 2>(v, lane & 4);  // 7 - i of half a row
    half_sum_step<0x4e, 1>(v, lane & 2);   // i ^ 2
    return v[0] + dpp_shift<0xb1, 0xf>(v[0]);  // i ^ 1
}

// Tile t of the product.  Eight p tiles share their q tiles before the next
// eight come.
__device__ __forceinline__ void pick_tile(int t, int p_tiles, int q_tiles, int& pt, int& qt, int& piece)
{
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
__global__ __launch_bounds__(S::kThreads, S::kWaves) void gated_product_kernel(Product<typename S::T> a)
{
    typedef typename S::T T;
    extern __shared__ char ring[];
    constexpr bool kGated = MODE == kFwd || MODE == kAgain;
    constexpr bool kPRows = MODE != kDw, kQRows = kGated;
    constexpr int kQTile = kGated ? S::BN / 2 : S::BN;  // output columns of a tile
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / S::WQ, wq = wave % S::WQ;
    const int col = lane & 31, q = lane >> 5;
    const int p_ld = kGated ? a.x_ld : 2 * a.Fp, q_ld = MODE == kDw ? a.x_ld : a.w_ld;

    // Workgroup b runs on XCD b mod 8; an XCD takes a contiguous run of tiles,
    // its workgroups take them in turn.
    const int xcd = blockIdx.x & 7, per = a.tiles >> 3, rem = a.tiles & 7, step = gridDim.x >> 3;
    const int first = xcd * per + min(xcd, rem) + (blockIdx.x >> 3);
    const int end = xcd * per + min(xcd, rem) + per + (xcd < rem ? 1 : 0);

    struct Tile {
        int64_t p0, m0;  // first p row; first contraction index of the piece
        int q0, K, pt, piece;
    };
    auto tile_of = [&](int t) __attribute__((always_inline)) {
        Tile r;
        int qt;
        pick_tile(t, a.p_tiles, a.q_tiles, r.pt, qt, r.piece);
        r.p0 = static_cast<int64_t>(r.pt) * S::BM;
        r.q0 = qt * kQTile;
        r.m0 = kGated ? 0 : r.piece * a.per;
        r.K = kGated ? a.C : static_cast<int>(min(a.per, (MODE == kDx ? 2 * static_cast<int64_t>(a.Fp) : a.rows) - r.m0));
        return r;
    };
    auto stages = [](int K) __attribute__((always_inline)) { return max(1, (K + S::BK - 1) / S::BK); };

    // The next stage to load: stage lk of tile lt.  Loads run ahead over the
    // ends of tiles, so a tile's first stages arrive during the epilogue of the
    // one before.
    Units<S, S::BM, kPRows> pu;
    Units<S, S::BN, kQRows> qu;
    int lt = first, lk = 0, lstages = 0, p_valid = 0, q_valid = 0;
    int to_up = 0;                           // stage of dx whose q rows are the first of Wu
    int left = 0, q_left = 0;                // contraction values from this stage on, and rows of the q source
    const T *p_src, *q_src, *q_src2;    // the stage's; q_src2: the other weight (gated: of the same stage, dx: from Fp on)
    const int64_t p_step = kPRows ? S::BK : static_cast<int64_t>(S::BK) * p_ld, q_step = kQRows ? S::BK : static_cast<int64_t>(S::BK) * q_ld;
    bool cut = false;                        // whether this stage's units are fewer than a whole one's
    auto whole_units = [&]() __attribute__((always_inline)) {
        pu.template set<false>(p_valid, p_ld);
        qu.template set<kQRows>(q_valid, q_ld);
    };
    auto cut_units = [&]() __attribute__((always_inline)) {
        cut = left < S::BK || q_left < S::BK;
        if (FAST && cut) {
            pu.cut(left);
            qu.cut(q_left);
        }
    };
    auto enter = [&]() __attribute__((always_inline)) {
        const Tile o = tile_of(lt);
        lk = 0;
        lstages = stages(o.K);
        left = o.K;
        const bool up = MODE == kDx && o.m0 >= a.Fp;  // the piece starts among the rows of Wu
        const int64_t q_row = MODE == kDx ? o.m0 - (up ? a.Fp : 0) : 0;
        q_left = MODE == kDx ? static_cast<int>(a.F - q_row) : o.K;
        to_up = MODE == kDx && !up ? static_cast<int>((a.Fp - o.m0) / S::BK) : 0x7fffffff;
        p_valid = static_cast<int>(kPRows ? min(static_cast<int64_t>(S::BM), a.rows - o.p0) : 2 * a.Fp - o.p0);
        q_valid = kQRows ? min(kQTile, a.F - o.q0) : a.C - o.q0;
        p_src = kPRows ? (kGated ? a.x : a.d) + o.p0 * p_ld + o.m0 : a.d + o.m0 * p_ld + o.p0;
        const int64_t q_at = kQRows ? static_cast<int64_t>(o.q0) * q_ld : o.q0;
        q_src = MODE == kDw ? a.x + o.m0 * q_ld + q_at : (up ? a.wu : a.wg) + q_row * q_ld + q_at;
        q_src2 = a.wu + q_at;
        whole_units();
        cut_units();
    };
    auto issue = [&](int i, char* st) __attribute__((always_inline)) {
        const bool is_p = i < S::kPLoads;
        const int j = is_p ? i : i - S::kPLoads;
        const T* src = is_p ? p_src : kQRows && qu.second(j) ? q_src2 : q_src;
        dma16(dma_rsrc(src, kAll), is_p ? pu.off[j] : qu.off[j], lds_addr(st + (is_p ? 0 : S::kPBytes) + (j * S::kThreads + wave * 64) * 16));
    };
    // Rows of any length and alignment pass through registers.
    uint4 held[FAST ? 1 : S::kLoads];
    auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (FAST ? 0 : S::kLoads); ++i) {
            const bool is_p = i < S::kPLoads;
            const int j = is_p ? i : i - S::kPLoads, have = is_p ? left : q_left;
            const T* src = is_p ? p_src : kQRows && qu.second(j) ? q_src2 : q_src;
            const int n = is_p ? pu.count(j, have, p_valid) : qu.count(j, have, q_valid);
            const bool ragged = (is_p ? kPRows : kQRows) ? have < S::BK && have % S::kUnit != 0 : (is_p ? p_valid % S::kUnit != 0 : q_valid % S::kUnit != 0);
            held[i] = unit_load<T>(make_rsrc(src, kAll), n > 0 ? (is_p ? pu.off[j] : qu.off[j]) : kOutside, ragged, n);
        }
    };
    auto put = [&](char* st) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (FAST ? 0 : S::kLoads); ++i) {
            const int j = i < S::kPLoads ? i : i - S::kPLoads;
            *reinterpret_cast<uint4*>(st + (i < S::kPLoads ? 0 : S::kPBytes) + (j * S::kThreads + threadIdx.x) * 16) = held[i];
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        if (++lk < lstages) {
            left -= S::BK;
            q_left -= S::BK;
            p_src += p_step;
            q_src += q_step;
            if (kQRows) q_src2 += q_step;
            if (MODE == kDx && lk == to_up) q_src = q_src2, q_left = a.F;  // Fp is a multiple of BK
            if (cut || left < S::BK || q_left < S::BK) {
                if (cut) whole_units();
                cut_units();
            }
            return;
        }
        lt += step;
        if (lt < end) {
            enter();
        } else if (FAST) {
            // no stage is left: the loads that still go out fetch nothing
            lstages = 0x7fffffff;
            pu.cut(0);
            qu.cut(0);
            left = q_left = 0x7fffffff;
            cut = false;
        }
    };

    f32x16 acc[S::TQ][S::TP];
    typename std::conditional<kPRows, RowFrag<S>, ColFrag<S, S::BM, S::TP>>::type pf(wp * S::TP);
    typename std::conditional<kQRows, RowFrag<S>, ColFrag<S, S::BN, S::TQ>>::type qf(wq * S::TQ);
    struct Frags {
        f32x4 q[S::TQ], p[S::TP];
    } frags[2];
    auto read_q = [&](Frags& f, const char* st, int kk, int i) __attribute__((always_inline)) {
        f.q[i] = qf.read((const lds_char*)st + S::kPBytes, wq * S::TQ + i, i, kk);
    };
    auto read_p = [&](Frags& f, const char* st, int kk, int j) __attribute__((always_inline)) {
        f.p[j] = pf.read((const lds_char*)st, wp * S::TP + j, j, kk);
    };
    constexpr int kSteps = S::kSteps;
    typedef std::integral_constant<int, 0> Zero;

    if (first >= end) return;
    enter();
    int cur = S::NS - 1;  // place of the stage being multiplied
    if constexpr (FAST) {
#pragma unroll 1
        for (int n = 0; n < S::NS - 1; ++n) {
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) issue(i, ring + n * S::kStage);
            advance();
        }
    } else {
        fetch();
        put(ring);
        advance();
        if (lt < end) fetch();
    }
    const char* here = nullptr;  // the stage being read, and the place of the one before it
    char* freed = nullptr;
    // Turns to the next stage.  It has landed for every wave after its own wait
    // and the barrier, and every wave has then read the one before into its
    // registers, so that one's place is free.
    auto turn_to_next = [&]() __attribute__((always_inline)) {
        if constexpr (FAST) {
            wait_vm_lds<(S::NS - 2) * S::kLoads>();
            barrier_no_fence();
        } else {
            __syncthreads();
            if (lt < end) {
                const int to = cur + 2 >= S::NS ? cur + 2 - S::NS : cur + 2;
                put(ring + to * S::kStage);
                advance();
                if (lt < end) fetch();
            }
        }
        freed = ring + cur * S::kStage;
        cur = cur + 1 == S::NS ? 0 : cur + 1;
        here = ring + cur * S::kStage;
    };
    // One step: the products of `f`, and between them the reads of the next
    // step's operands (`next` of stage `here`) and part `part` of the loads that
    // fill the freed place, one at a time: a wave issues in order, and a bunch
    // of other instructions leaves the matrix unit without work.
    auto step_of = [&](auto turn, Frags& f, Frags& n, int next, auto part) __attribute__((always_inline)) {
        constexpr int kProducts = S::TP * S::TQ, kReads = S::TP + S::TQ;
        constexpr int kFrom = part() * S::kLoads / kSteps, kPart = FAST ? (part() + 1) * S::kLoads / kSteps - kFrom : 0;
        constexpr int kItems = kReads + kPart + 1;
        auto item = [&](int x) __attribute__((always_inline)) {
            if (x < S::TQ) read_q(n, here, next, x);
            else if (x < kReads) read_p(n, here, next, x - S::TQ);
            else if (x < kReads + kPart) issue(kFrom + x - kReads, freed);
            else if (FAST && part() + 1 == kSteps) advance();
        };
#pragma unroll
        for (int m = 0; m < kProducts; ++m) {
            const int i = m / S::TP, j = m % S::TP;
            acc[i][j] = multiply<T>(f.q[i], f.p[j], acc[i][j]);
            if (m == 0 && turn()) turn_to_next();
#pragma unroll
            for (int x = m * kItems / kProducts; x < (m + 1) * kItems / kProducts; ++x) item(x);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // The biases of a tile's columns (both halves), a thread one of them: on
    // their way during the epilogue of the tile before.
    float bias = 0.f;
    auto load_bias = [&](int t) __attribute__((always_inline)) {
        if (!kGated || !a.bg || threadIdx.x >= S::BN) return;
        const int f = tile_of(t).q0 + threadIdx.x % kQTile;
        bias = 0.f;
        if (f < a.F) bias = load_f((threadIdx.x < kQTile ? a.bg : a.bu) + f);
    };
    load_bias(first);
    float* biases = reinterpret_cast<float*>(ring + S::NS * S::kStage);

    for (int t = first; t < end; t += step) {
        const Tile o = tile_of(t);
        const int nk = stages(o.K);
        const bool biased = kGated && a.bg;
        if (biased && threadIdx.x < S::BN) biases[threadIdx.x] = bias;
        turn_to_next();
#pragma unroll
        for (int i = 0; i < S::TQ; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
                if (biased) b = *reinterpret_cast<const float4*>(biases + (i & 1) * kQTile + (wq * (S::TQ / 2) + (i >> 1)) * 32 + 8 * v + 4 * q);
#pragma unroll
                for (int j = 0; j < S::TP; ++j) {
                    acc[i][j][4 * v] = b.x;
                    acc[i][j][4 * v + 1] = b.y;
                    acc[i][j][4 * v + 2] = b.z;
                    acc[i][j][4 * v + 3] = b.w;
                }
            }
        if constexpr (FAST) {
#pragma unroll
            for (int i = 0; i < S::kLoads / kSteps; ++i) issue(i, freed);
        }
#pragma unroll
        for (int i = 0; i < S::TQ; ++i) read_q(frags[0], here, 0, i);
#pragma unroll
        for (int j = 0; j < S::TP; ++j) read_p(frags[0], here, 0, j);
        static_assert(kSteps == 2 || kSteps == 4, "the next stage's operands take the first place again");
        auto first_steps = [&]() __attribute__((always_inline)) {
            step_of(std::false_type{}, frags[0], frags[1], 1, std::integral_constant<int, 1>{});
            if constexpr (kSteps == 4) {
                step_of(std::false_type{}, frags[1], frags[0], 2, std::integral_constant<int, 2>{});
                step_of(std::false_type{}, frags[0], frags[1], 3, std::integral_constant<int, 3>{});
            }
        };
        // Ahead of the other wave of the SIMD while it is in its epilogue: the
        // matrix unit is free then, and the epilogue fills the gaps (100352
        // rows, 256 -> 2 x 1024: 185 -> 173 us).
        __builtin_amdgcn_s_setprio(2);
        for (int kt = 1; kt < nk; ++kt) {
            first_steps();
            // The last step's operands are in registers: on to the next stage,
            // whose first operands arrive during this step.
            step_of(std::true_type{}, frags[1], frags[0], 0, Zero{});
        }
        first_steps();
#pragma unroll
        for (int m = 0; m < S::TP * S::TQ; ++m)
            acc[m / S::TP][m % S::TP] = multiply<T>(frags[1].q[m / S::TP], frags[1].p[m % S::TP], acc[m / S::TP][m % S::TP]);
        // Every wave is done with the last stage, whose place the outputs pass
        // through; it is filled again after the next turn.
        wait_vm_lds<63>();
        barrier_no_fence();
        __builtin_amdgcn_s_setprio(0);
        if (t + step < end) load_bias(t + step);
        char* turn = const_cast<char*>(here) + wave * S::kWaveLds;

        // A lane holds columns 8v + 4q + {0..3} of a q tile and p row `col`.
        if constexpr (kGated) {
            // A step takes 32 rows and 32 columns.  The activation of eight
            // values at a time: enough for its latencies, few enough that the
            // accumulators stay in registers.
            constexpr int M = S::TQ / 2, UO = 32 / S::kUnit;  // UO: units of 32 columns
            const int f0 = o.q0 + wq * M * 32;                // the wave's first column
            float tg[M], tu[M];                               // column sums
#pragma unroll
            for (int m = 0; m < M; ++m) tg[m] = tu[m] = 0.f;
            uint4 dh[UO / 2];
            auto load_dh = [&](int s) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < UO / 2; ++i) {
                    const int64_t r0 = o.p0 + (wp * S::TP + s / M) * 32;
                    const int r = (i * 64 + lane) / UO, at = lane % UO * S::kUnit, fs = f0 + s % M * 32, n = a.F - fs - at;
                    const rsrc_t in = make_rsrc(a.dh + r0 * a.F + fs, kAll);
                    const bool on = r < a.rows - r0 && n > 0;
                    dh[i] = unit_load<T>(in, on ? static_cast<uint32_t>(r * a.F + at) * S::E : kOutside, fs + 32 > a.F && a.F % S::kUnit != 0, on ? n : 0);
                }
            };
            // Columns 8v + 4q + {0..3} of this lane's row.
            auto lay = [&](char* to, int v, const float* w) __attribute__((always_inline)) {
                if constexpr (S::E == 2)
                    *reinterpret_cast<uint2*>(to + turn_at<4>(col, v) + 8 * q) = make_uint2(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]));
                else
                    *reinterpret_cast<float4*>(to + turn_at<8>(col, 2 * v + q)) = make_float4(w[0], w[1], w[2], w[3]);
            };
            if constexpr (MODE == kAgain) load_dh(0);
#pragma unroll
            for (int s = 0; s < S::TP * M; ++s) {
                __builtin_amdgcn_sched_barrier(0);
                const int j = s / M, m = s % M;
                const int64_t r0 = o.p0 + (wp * S::TP + j) * 32;
                const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.rows - r0));
                const int fs = f0 + m * 32;
                const f32x16 &g = acc[2 * m][j], &u = acc[2 * m + 1][j];
                if constexpr (MODE == kFwd) {
                    if (a.saved) {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const f32x16& w = n ? u : g;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                *reinterpret_cast<float4*>(turn + turn_at<8>(col, 2 * v + q)) = make_float4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                            wave_order();
                            turn_out<8>(turn, a.saved + r0 * 2 * a.F + (n ? a.F : 0) + fs, 2u * a.F, rows, a.F - fs);
                            wave_order();
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float h[8];
                        with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = act_value<kind()>(g[8 * half + e]) * u[8 * half + e];
                        });
                        lay(turn, 2 * half, h);
                        lay(turn, 2 * half + 1, h + 4);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    wave_order();
                    turn_out<UO>(turn, a.h + r0 * a.F + fs, a.F, rows, a.F - fs);
                } else {
                    char* other = turn + (S::E == 2 ? 2048 : 0);
#pragma unroll
                    for (int i = 0; i < UO / 2; ++i) *reinterpret_cast<uint4*>(turn + turn_at<UO>((i * 64 + lane) / UO, lane % UO)) = dh[i];
                    wave_order();
                    if (s + 1 < S::TP * M) load_dh(s + 1);
                    float dg[16], du[16];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float h[8];
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            if constexpr (S::E == 2) {
                                const uint2 raw = *reinterpret_cast<const uint2*>(turn + turn_at<4>(col, 2 * half + v) + 8 * q);
                                h[4 * v] = __uint_as_float(raw.x << 16), h[4 * v + 1] = __uint_as_float(raw.x & 0xffff0000u);
                                h[4 * v + 2] = __uint_as_float(raw.y << 16), h[4 * v + 3] = __uint_as_float(raw.y & 0xffff0000u);
                            } else {
                                const float4 raw = *reinterpret_cast<const float4*>(turn + turn_at<8>(col, 2 * (2 * half + v) + q));
                                h[4 * v] = raw.x, h[4 * v + 1] = raw.y, h[4 * v + 2] = raw.z, h[4 * v + 3] = raw.w;
                            }
                        }
                        with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const ActPair p = act_pair<kind()>(g[8 * half + e]);
                                dg[8 * half + e] = h[e] * u[8 * half + e] * p.d;
                                du[8 * half + e] = h[e] * p.v;
                            }
                        });
#pragma unroll
                        for (int v = 2 * half; v < 2 * half + 2; ++v) {
                            lay(turn, v, dg + 4 * v);  // where this lane's dh was
                            if (S::E == 2) lay(other, v, du + 4 * v);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    wave_order();
                    // the columns up to Fp too: their dh is 0, and so are they
                    T* d = a.d_out + r0 * 2 * a.Fp + fs;
                    turn_out<UO>(turn, d, 2u * a.Fp, rows, a.Fp - fs);
                    if constexpr (S::E == 4) {
                        wave_order();
#pragma unroll
                        for (int v = 0; v < 4; ++v) lay(other, v, du + 4 * v);
                        wave_order();
                    }
                    turn_out<UO>(other, d + a.Fp, 2u * a.Fp, rows, a.Fp - fs);
                    if (a.sums) {
                        tg[m] += half_sum16(dg, lane);
                        tu[m] += half_sum16(du, lane);
                    }
                }
                wave_order();
            }
            if (MODE == kAgain && a.sums) {
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int which = half_sum_of(lane);
                    const int f = f0 + m * 32 + 8 * (which >> 2) + 4 * q + (which & 3);
                    if ((lane & 1) == 0 && f < a.Fp) {
                        float* row = a.sums + static_cast<int64_t>(o.pt * S::WP + wp) * 2 * a.Fp;
                        row[f] = tg[m];
                        row[a.Fp + f] = tu[m];
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < S::TP; ++j) {
                // 32 rows of dx, or (Fp is a multiple of 32) of dWg or dWu
                const int64_t r0 = o.p0 + (wp * S::TP + j) * 32;
                const int c0 = o.q0 + wq * S::TQ * 32;
                T* out = a.out;
                float* part = nullptr;
                int64_t f = r0;
                int rows;
                if (MODE == kDx) {
                    rows = static_cast<int>(min(static_cast<int64_t>(32), a.rows - r0));
                    if (a.part) part = a.part + (o.piece * a.rows + r0) * a.C;
                } else {
                    const bool up = r0 >= a.Fp;
                    f -= up ? a.Fp : 0;
                    rows = r0 < 2 * a.Fp ? static_cast<int>(min(static_cast<int64_t>(32), a.F - f)) : 0;
                    out = up ? a.out2 : a.out;
                    if (a.part) part = a.part + ((static_cast<int64_t>(o.piece) * 2 + (up ? 1 : 0)) * a.F + f) * a.C;
                }
                if (S::E == 4 || part) {
#pragma unroll
                    for (int i = 0; i < S::TQ; ++i) {
                        __builtin_amdgcn_sched_barrier(0);
                        const f32x16& w = acc[i][j];
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            *reinterpret_cast<float4*>(turn + turn_at<8>(col, 2 * v + q)) = make_float4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                        wave_order();
                        float* to = part;
                        if constexpr (S::E == 4) {
                            if (!to && out) to = out + f * a.C;
                        }
                        if (to) turn_out<8>(turn, to + c0 + i * 32, a.C, rows, a.C - c0 - i * 32);
                        wave_order();
                    }
                } else if constexpr (S::E == 2) {
#pragma unroll
                    for (int i = 0; i < S::TQ; i += 2) {
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const f32x16& w = acc[i + n][j];
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                *reinterpret_cast<uint2*>(turn + turn_at<8>(col, n * 4 + v) + 8 * q) = make_uint2(pack_bf16x2(w[4 * v], w[4 * v + 1]), pack_bf16x2(w[4 * v + 2], w[4 * v + 3]));
                        }
                        wave_order();
                        if (out) turn_out<8>(turn, out + f * a.C + c0 + i * 32, a.C, rows, a.C - c0 - i * 32);
                        wave_order();
                    }
                }
            }
        }
    }
    if constexpr (FAST) wait_vm_lds<0>();  // no load may arrive in LDS that is no longer this workgroup's
}

// Few rows: the layer is a stream over its weights.  A workgroup takes 16
// hidden channels (16 rows of Wg and of Wu), its waves share the contraction
// in pieces, NP groups of 16 rows of x ride along, and the waves' sums are
// added in order.  MODE kFwd: h; kAgain: dg and du, and their column sums.  A 16-byte load a lane is one 16x16x32 instruction in bf16,
// four 16x16x4 in fp32.
constexpr int kFewWaves = 8;
template <typename T>
__device__ __forceinline__ f32x4 multiply16(uint4 w, uint4 x, f32x4 acc)
{
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    } else {
        const f32x4 a = __builtin_bit_cast(f32x4, w), b = __builtin_bit_cast(f32x4, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
        return acc;
    }
}
template <typename T, int MODE, int NP, bool FAST>
__global__ __launch_bounds__(kFewWaves * 64) void gated_few_rows_kernel(Product<T> a)
{
    constexpr int kUnit = 16 / sizeof(T), kLoad = 4 * kUnit, kPiece = 2 * kLoad;  // contraction values of a load, of a piece
    __shared__ f32x4 sums[kFewWaves][2][NP][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 15, ku = (lane >> 4) * kUnit;
    const int f0 = blockIdx.x * 16;
    const int64_t fr = min(f0 + row, a.F - 1);  // past F (up to Fp): not used
    const T *wg = a.wg + fr * a.w_ld, *wu = a.wu + fr * a.w_ld;
    const T* x[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) x[j] = a.x + min(static_cast<int64_t>(j * 16 + row), a.rows - 1) * a.x_ld;
    f32x4 g[NP], u[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) g[j] = u[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // The first values of a row's last, cut unit by elements.
    auto load = [&](const T* p, int k) __attribute__((always_inline)) {
        if (k >= a.C) return make_uint4(0, 0, 0, 0);
        if (FAST) return *reinterpret_cast<const uint4*>(p + k);
        const int n = a.C - k;
        if (n >= kUnit) return load16_any(p + k);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kUnit; ++e) {
            const T v = p[k + min(e, n - 1)];
            if constexpr (sizeof(T) == 2) w[e >> 1] |= (e < n ? static_cast<uint32_t>(v) : 0u) << (16 * (e & 1));
            else w[e] = e < n ? __float_as_uint(v) : 0u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    constexpr int U = NP == 1 ? 2 : 1;  // pieces in flight
    for (int k0 = wave * kPiece; k0 < a.C; k0 += kFewWaves * kPiece * U) {
        uint4 vg[U][2], vu[U][2], vx[U][2][NP];
#pragma unroll
        for (int t = 0; t < U; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = k0 + t * kFewWaves * kPiece + s * kLoad + ku;
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
                    g[j] = multiply16<T>(vg[t][s], vx[t][s][j], g[j]);
                    u[j] = multiply16<T>(vu[t][s], vx[t][s][j], u[j]);
                }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        sums[wave][0][j][lane] = g[j];
        sums[wave][1][j][lane] = u[j];
    }
    __syncthreads();
    // value (p, f): lane (f / 4) * 16 + p of a group, element f % 4
    __shared__ float down[MODE == kAgain ? 2 : 1][MODE == kAgain ? NP * 16 : 1][16];
    for (int idx = threadIdx.x; idx < NP * 256; idx += kFewWaves * 64) {
        const int f = idx & 15, p = idx >> 4;
        const bool on = p < a.rows && f0 + f < a.F;
        const int at = (f >> 2) * 16 + (p & 15);
        float gv = 0.f, uv = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) {
            gv += reinterpret_cast<const float*>(&sums[w][0][p >> 4][at])[f & 3];
            uv += reinterpret_cast<const float*>(&sums[w][1][p >> 4][at])[f & 3];
        }
        if (a.bg && on) gv += load_f(a.bg + f0 + f), uv += load_f(a.bu + f0 + f);
        if constexpr (MODE == kFwd) {
            if (!on) continue;
            if (a.saved) {
                a.saved[static_cast<int64_t>(p) * 2 * a.F + f0 + f] = gv;
                a.saved[static_cast<int64_t>(p) * 2 * a.F + a.F + f0 + f] = uv;
            }
            store_f(a.h + static_cast<int64_t>(p) * a.F + f0 + f, act_value(a.act, gv) * uv);
        } else {
            // the columns up to Fp too: zeros
            const float dh = on ? load_f(a.dh + static_cast<int64_t>(p) * a.F + f0 + f) : 0.f;
            const ActPair t = act_pair(a.act, gv);
            const float dg = on ? dh * uv * t.d : 0.f, du = on ? dh * t.v : 0.f;
            if (p < a.rows) {
                T* d = a.d_out + static_cast<int64_t>(p) * 2 * a.Fp + f0 + f;
                store_f(d, dg);
                store_f(d + a.Fp, du);
            }
            down[0][p][f] = dg;
            down[1][p][f] = du;
        }
    }
    if constexpr (MODE == kAgain) {
        if (!a.sums) return;
        __syncthreads();
        if (threadIdx.x < 32) {
            const int f = threadIdx.x & 15, half = threadIdx.x >> 4;
            float t = 0.f;
            for (int p = 0; p < NP * 16; ++p) t += down[half][p][f];
            a.sums[static_cast<int64_t>(half) * a.Fp + f0 + f] = t;
        }
    }
}

// Tiles of either type; a stage is 64 or 128 bytes of contraction values.
template <typename T>
struct Tiles {
    typedef Shape<bf16_t, 2, 2, 4, 4, 32, 4> Wide;   // 256 x 256, one workgroup a CU
    typedef Shape<bf16_t, 2, 2, 2, 4, 32, 3> Big;    // 128 x 256, two
    typedef Shape<bf16_t, 2, 2, 2, 2, 64, 2> Small;  // 128 x 128
    typedef Shape<bf16_t, 4, 1, 1, 2, 64, 4> Thin;   // 128 x 64, a deep ring
};
template <>
struct Tiles<float> {
    typedef Shape<float, 2, 2, 1, 2, 32, 2> Small;  // 64 x 128
    typedef Small Wide, Big;
    typedef Shape<float, 4, 1, 1, 2, 32, 2> Thin;   // 128 x 64
};

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int64_t tiles(int64_t n, int t) { return (n + t - 1) / t; }

template <typename S, int MODE, bool FAST>
hipError_t run(Product<typename S::T>& k, int64_t p, int64_t q, int pieces, hipStream_t s)
{
    const int64_t pt = tiles(p, S::BM), qt = tiles(q, S::BN), n = pt * qt * pieces;
    if (n >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    k.p_tiles = static_cast<int>(pt);
    k.q_tiles = static_cast<int>(qt);
    k.tiles = static_cast<int>(n);
    auto kernel = gated_product_kernel<S, MODE, FAST>;
    static std::atomic<bool> ready{false};
    if (S::kLds > 65536 && !ready.load(std::memory_order_acquire)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
        if (e != hipSuccess) return e;
        ready.store(true, std::memory_order_release);
    }
    // as many workgroups as the device holds at once, the same number on each XCD
    const int64_t hold = std::max(8, device_cu_count() * S::kPerCu / 8 * 8);
    return launch(kernel, dim3(static_cast<unsigned>(std::min<int64_t>((n + 7) / 8 * 8, hold))), dim3(S::kThreads), S::kLds, s, k);
}

// Which tile: the one whose rounds take the least time.  A round is one tile in
// every place of the device, and takes the tile's products at the rate that the
// tile reaches plus its epilogue (us; what the other workgroup of a CU does not
// hide of it).  Rates (TFLOP/s) and epilogues as measured: 256 x 256 tiles
// reach 1150, have half the loads and LDS reads for a product, and nothing
// beside their epilogue; 128 x 256 1050, 128 x 128 750 (all bf16); fp32's
// instructions leave time for every load, 64 x 128 reach 105, 128 x 256 no more.
// fp32 has tiles of 64 x 128 and 128 x 64 (1 to 2 % slower), and takes those
// that cover the output with fewer, if by 3 %: 1001 rows, 190 -> 2 x 517, training
// step: 61 us, 69 with 64 x 128 alone; 20000 rows, 64 -> 2 x 256: 93 and 103.
//
// The forward product's sum is not cut into pieces.  Where its small tiles are
// fewer than the CUs it is a stream over the weights, bound by the loads in
// flight: the thin tile has twice the workgroups and three stages of loads
// ahead instead of one (128 rows, 4096 -> 2 x 8192: 34 us, 28 the weights' stream).
enum class Tile { kThin, kSmall, kBig, kWide };
template <typename S>
double tile_us(int64_t K, double rate, double epilogue)
{
    return 2e-6 * S::BM * S::BN * static_cast<double>(K) / rate * S::kPerCu * device_cu_count() + epilogue;
}
template <typename S>
double rounds_us(int64_t n, int64_t K, double rate, double epilogue)
{
    const int64_t places = S::kPerCu * static_cast<int64_t>(device_cu_count());
    return static_cast<double>((n + places - 1) / places) * tile_us<S>(K, rate, epilogue);
}
// Calls f with the tile's shape.
template <typename T, typename F>
auto with_tile(Tile t, F f)
{
    if (t == Tile::kWide) return f(typename Tiles<T>::Wide{});
    if (t == Tile::kBig) return f(typename Tiles<T>::Big{});
    if (t == Tile::kThin) return f(typename Tiles<T>::Thin{});
    return f(typename Tiles<T>::Small{});
}
// The time of `pieces` products over K values each, by tile.
template <typename T>
double product_us(Tile t, int64_t p, int64_t q, int64_t K, int pieces)
{
    typedef Tiles<T> X;
    if constexpr (sizeof(T) == 4)
        return with_tile<T>(t, [&](auto shape) { return rounds_us<decltype(shape)>(tiles(p, shape.BM) * tiles(q, shape.BN) * pieces, K, 105, 1); });
    if (t == Tile::kWide) return rounds_us<typename X::Wide>(tiles(p, X::Wide::BM) * tiles(q, X::Wide::BN) * pieces, K, 1150, 10);
    if (t == Tile::kBig) return rounds_us<typename X::Big>(tiles(p, X::Big::BM) * tiles(q, X::Big::BN) * pieces, K, 1050, 4);
    return rounds_us<typename X::Small>(tiles(p, X::Small::BM) * tiles(q, X::Small::BN) * pieces, K, 750, 2);
}
template <typename T>
Tile pick(int64_t p, int64_t q, int64_t K, int pieces = 1)
{
    typedef Tiles<T> X;
    if (sizeof(T) == 4) {
        const int64_t thin = tiles(p, X::Thin::BM) * tiles(q, X::Thin::BN), small = tiles(p, X::Small::BM) * tiles(q, X::Small::BN);
        return 33 * thin < 32 * small ? Tile::kThin : Tile::kSmall;
    }
    Tile best = Tile::kSmall;
    for (Tile t : {Tile::kBig, Tile::kWide})
        if (product_us<T>(t, p, q, K, pieces) < product_us<T>(best, p, q, K, pieces)) best = t;
    return best;
}
template <typename T>
Tile pick_gated(const GatedArgs& a)
{
    typedef typename Tiles<T>::Small Small;
    const int64_t q = 2 * static_cast<int64_t>(a.F);
    if (sizeof(T) == 2 && tiles(a.rows, Small::BM) * tiles(q, Small::BN) < device_cu_count()) return Tile::kThin;
    return pick<T>(a.rows, q, a.C);
}
// Partial rows of the column sums of `rows` rows: one for each wave's rows.
template <typename T>
int64_t sum_rows(int64_t rows, Tile t)
{
    return with_tile<T>(t, [&](auto shape) { return tiles(rows, shape.BM) * shape.WP; });
}

// Pieces of a sum over K for a p x q output, none under `least` values, a whole
// number of stages each, and the tile: where the rounds of the pieces and the
// stream over their partials (written and read, 3.5 TB/s, and their sums' launch)
// take the least time.
struct Split {
    int64_t per;
    int pieces;
    Tile tile;
};
template <typename T>
Split split(int64_t p, int64_t q, int64_t K, int64_t least)
{
    Split best{std::max<int64_t>(64, (K + 63) / 64 * 64), 1, pick<T>(p, q, K)};
    double time = product_us<T>(best.tile, p, q, K, 1);
    for (int64_t n = 2; n <= K / least && n <= 64; ++n) {
        const int64_t per = (tiles(K, static_cast<int>(n)) + 63) / 64 * 64;
        const int pieces = static_cast<int>((K + per - 1) / per);
        const double sums = 3 + 8.0 * pieces * p * q / 3.5e6;
        for (Tile t : {Tile::kSmall, Tile::kBig, Tile::kWide}) {
            if (sizeof(T) == 4) t = pick<T>(p, q, per);
            const double us = product_us<T>(t, p, q, per, pieces) + sums;
            if (us < time) time = us, best = Split{per, pieces, t};
        }
    }
    return best;
}

template <int MODE, typename T>
hipError_t run_tiles(Product<T>& k, int64_t p, int64_t q, int pieces, Tile t, bool fast, hipStream_t s)
{
    typedef Tiles<T> X;
    if constexpr (sizeof(T) == 2)
        if (t == Tile::kWide && fast) return run<typename X::Wide, MODE, true>(k, p, q, pieces, s);
    if constexpr (sizeof(T) == 4 || MODE == kFwd || MODE == kAgain)
        if (t == Tile::kThin) return fast ? run<typename X::Thin, MODE, true>(k, p, q, pieces, s) : run<typename X::Thin, MODE, false>(k, p, q, pieces, s);
    if constexpr (sizeof(T) == 2)
        if (t != Tile::kSmall) return fast ? run<typename X::Big, MODE, true>(k, p, q, pieces, s) : run<typename X::Big, MODE, false>(k, p, q, pieces, s);
    return fast ? run<typename X::Small, MODE, true>(k, p, q, pieces, s) : run<typename X::Small, MODE, false>(k, p, q, pieces, s);
}

constexpr int64_t kFewRows = 64;

template <typename T>
Product<T> product(const GatedArgs& a)
{
    Product<T> k{};
    k.x = static_cast<const T*>(a.x);
    k.wg = static_cast<const T*>(a.wg);
    k.wu = static_cast<const T*>(a.wu);
    k.bg = static_cast<const T*>(a.bg);
    k.bu = static_cast<const T*>(a.bu);
    k.dh = static_cast<const T*>(a.dh);
    k.rows = a.rows;
    k.C = a.C;
    k.F = a.F;
    k.act = a.act;
    k.x_ld = k.w_ld = a.C;
    return k;
}

// Rows of a length that is no whole number of 16-byte units cannot go straight
// to LDS, and passing them through registers takes the products to a third of
// their rate.  So x and the weights are copied to rows with zeros behind them
// first, which costs a launch and their bytes twice.  Training step, with
// copies and without: 2000 rows, 1001 -> 2 x 3001: 176 and 385 us; 500 rows,
// 101 -> 2 x 333: 49 and 85; 5 rows, 1001 -> 2 x 3001: 48 and 63.  The forward product alone (rows of x and weights
// only, no columns) is slowed less: 42 and 52 us, 11 and 7, 1000 rows, 301 ->
// 2 x 733: 14 and 10; it copies from kPadForward products on.
constexpr int64_t kPadForward = int64_t(1) << 30;
template <typename T>
struct Padded {
    int ld = 0;  // values; 0: no copies
    size_t bytes = 0;
    Padded(int64_t rows, int C, int F, bool forward)
    {
        if (C % (16 / sizeof(T)) == 0 || rows == 0 || (forward && (rows <= kFewRows || rows * F * C < kPadForward))) return;
        ld = (C + 63) / 64 * 64;
        bytes = round256((static_cast<size_t>(rows) + 2 * static_cast<size_t>(F)) * ld * sizeof(T));
    }
};
template <typename T>
struct PadArgs {
    const T* src[3];
    T* dst[3];
    int64_t rows[3];
    int C, ld;
};
// A wave a row; lanes past the row write zeros.
template <typename T>
__global__ __launch_bounds__(256) void gated_pad_kernel(PadArgs<T> a)
{
    constexpr int kUnit = 16 / sizeof(T);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T* src = a.src[blockIdx.y];
    T* dst = a.dst[blockIdx.y];
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + wave; r < a.rows[blockIdx.y]; r += static_cast<int64_t>(gridDim.x) * 4)
        for (int c = lane * kUnit; c < a.ld; c += 64 * kUnit) {
            const T* p = src + r * a.C + c;
            const int n = a.C - c;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (n >= kUnit) {
                v = load16_any(p);
            } else if (n > 0) {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < kUnit; ++e)
                    if (e < n) {
                        if constexpr (sizeof(T) == 2) w[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
                        else w[e] = __float_as_uint(p[e]);
                    }
                v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4*>(dst + r * a.ld + c) = v;
        }
}
// Copies x and the weights to `at` and points k to the copies.
template <typename T>
hipError_t pad(Product<T>& k, int ld, char* at, hipStream_t s)
{
    PadArgs<T> a{};
    a.C = k.C;
    a.ld = ld;
    const T* src[3] = {k.x, k.wg, k.wu};
    T* dst = reinterpret_cast<T*>(at);
    for (int i = 0; i < 3; ++i) {
        a.src[i] = src[i];
        a.dst[i] = dst;
        a.rows[i] = i ? k.F : k.rows;
        dst += a.rows[i] * ld;
    }
    const int64_t most = std::max<int64_t>(k.rows, k.F);
    const hipError_t e = launch(gated_pad_kernel<T>, dim3(static_cast<unsigned>(std::min<int64_t>((most + 3) / 4, 8 * device_cu_count())), 3), dim3(256), 0, s, a);
    k.x = a.dst[0];
    k.wg = a.dst[1];
    k.wu = a.dst[2];
    k.x_ld = k.w_ld = ld;
    return e;
}

constexpr int64_t kLeastRows = 256, kLeastHidden = 512;  // of a piece of dW's sum, of dx's

template <typename T>
GatedPlan gated_plan(int64_t rows, int C, int F)
{
    GatedPlan p{};
    p.Fp = (F + 63) / 64 * 64;
    const int64_t dp = 2 * static_cast<int64_t>(p.Fp), least = sizeof(T) == 2 ? 1 : 4;
    const Split w = split<T>(dp, C, rows, kLeastRows / least), x = split<T>(rows, C, dp, kLeastHidden / least);
    p.per = w.per;
    p.pieces = w.pieces;
    p.tile = static_cast<int>(w.tile);
    p.x_per = x.per;
    p.x_pieces = x.pieces;
    p.x_tile = static_cast<int>(x.tile);
    int64_t chunk;
    p.sum_rows = static_cast<int>(std::max<int64_t>(gated_kept_chunks(rows, p.Fp, &chunk), std::max(sum_rows<T>(rows, Tile::kSmall), sum_rows<T>(rows, Tile::kThin))));
    p.d_bytes = round256(static_cast<size_t>(rows) * 2 * p.Fp * sizeof(T));
    p.sum_bytes = round256(static_cast<size_t>(p.sum_rows) * 2 * p.Fp * 4);
    p.pad_bytes = Padded<T>(rows, C, F, false).bytes;
    p.x_bytes = p.x_pieces > 1 ? round256(static_cast<size_t>(p.x_pieces) * rows * C * 4) : 0;
    p.w_bytes = p.pieces > 1 ? round256(static_cast<size_t>(p.pieces) * 2 * F * C * 4) : 0;
    return p;
}

template <int MODE, typename T>
hipError_t few_rows(const Product<T>& k, int columns, bool fast, hipStream_t s)
{
    const dim3 grid((columns + 15) / 16), block(kFewWaves * 64);
    if (k.rows <= 16) return launch(fast ? gated_few_rows_kernel<T, MODE, 1, true> : gated_few_rows_kernel<T, MODE, 1, false>, grid, block, 0, s, k);
    if (k.rows <= 32) return launch(fast ? gated_few_rows_kernel<T, MODE, 2, true> : gated_few_rows_kernel<T, MODE, 2, false>, grid, block, 0, s, k);
    return launch(fast ? gated_few_rows_kernel<T, MODE, 4, true> : gated_few_rows_kernel<T, MODE, 4, false>, grid, block, 0, s, k);
}

template <typename T>
hipError_t gated_fwd(const GatedArgs& a, hipStream_t s)
{
    Product<T> k = product<T>(a);
    k.h = static_cast<T*>(a.h);
    k.saved = a.saved;
    bool fast = a.C % (16 / sizeof(T)) == 0 && aligned(a.x) && aligned(a.wg) && aligned(a.wu);
    if (a.rows <= kFewRows) return few_rows<kFwd>(k, a.F, fast, s);
    const Padded<T> padded(a.rows, a.C, a.F, true);
    if (padded.ld && a.workspace) {
        const ArmedEvents armed = armed_events();
        armed_events() = ArmedEvents{armed.start, nullptr};
        const hipError_t e = pad(k, padded.ld, static_cast<char*>(a.workspace), s);
        armed_events() = ArmedEvents{nullptr, armed.stop};
        if (e != hipSuccess) {
            armed_events() = ArmedEvents{nullptr, nullptr};
            return e;
        }
        fast = true;
    }
    return run_tiles<kFwd>(k, a.rows, 2 * static_cast<int64_t>(a.F), 1, pick_gated<T>(a), fast, s);
}

template <typename T>
size_t gated_fwd_workspace(int64_t rows, int C, int F) { return Padded<T>(rows, C, F, true).bytes; }

template <typename T>
hipError_t gated_bwd(const GatedArgs& a, hipStream_t s)
{
    constexpr int kUnit = 16 / sizeof(T), kType = sizeof(T) == 2;
    const GatedPlan p = gated_plan<T>(a.rows, a.C, a.F);
    char* ws = static_cast<char*>(a.workspace);
    T* d = reinterpret_cast<T*>(ws);
    float* sums = a.dbg || a.dbu ? reinterpret_cast<float*>(ws + p.d_bytes) : nullptr;
    float* x_part = p.x_pieces > 1 && a.dx ? reinterpret_cast<float*>(ws + p.d_bytes + p.sum_bytes) : nullptr;
    float* w_part = p.pieces > 1 ? reinterpret_cast<float*>(ws + p.d_bytes + p.sum_bytes + p.x_bytes) : nullptr;
    // What comes after dg and du, to know the call's last launch.
    const bool dx = a.dx && a.rows > 0, weights = a.dwg || a.dwu, added = (dx && x_part) || (weights && w_part) || sums;
    CallEvents events;
    hipError_t e = hipSuccess;
    int summed = 0;
    Product<T> k = product<T>(a);
    k.Fp = p.Fp;
    const Padded<T> padded(a.rows, a.C, a.F, false);
    if (padded.ld) {
        events.next(false);
        e = pad(k, padded.ld, ws + p.d_bytes + p.sum_bytes + p.x_bytes + p.w_bytes, s);
        if (e != hipSuccess) return e;
    }
    const bool whole = padded.ld || a.C % kUnit == 0;  // rows are whole units
    if (a.rows > 0) {
        events.next(!dx && !weights && !added);
        if (a.saved) {
            int64_t chunk;
            summed = gated_kept_chunks(a.rows, p.Fp, &chunk);
            e = launch_gated_kept(a, d, sums, p.Fp, summed, chunk, kType, s);
        } else {
            k.d_out = d;
            k.sums = sums;
            const bool fast = whole && aligned(k.x) && aligned(k.wg) && aligned(k.wu);
            if (a.rows <= kFewRows) {
                summed = 1;
                e = few_rows<kAgain>(k, p.Fp, fast, s);
            } else {
                Tile t = pick_gated<T>(a);
                if (t == Tile::kWide && !fast) t = Tile::kBig;
                summed = static_cast<int>(sum_rows<T>(a.rows, t));
                e = run_tiles<kAgain>(k, a.rows, 2 * static_cast<int64_t>(p.Fp), 1, t, fast, s);  // the columns up to Fp too
            }
        }
        if (e != hipSuccess) return e;
        k.d = d;
        if (dx) {
            k.out = static_cast<T*>(a.dx);
            k.part = x_part;
            k.per = p.x_per;
            events.next(!weights && !added);
            e = run_tiles<kDx>(k, a.rows, a.C, p.x_pieces, static_cast<Tile>(p.x_tile),
                               whole && aligned(k.wg) && aligned(k.wu), s);
            if (e != hipSuccess) return e;
        }
    }
    if (weights) {
        k.d = d;
        k.out = static_cast<T*>(a.dwg);
        k.out2 = static_cast<T*>(a.dwu);
        k.part = w_part;
        k.per = p.per;
        events.next(!added);
        const int64_t dp = 2 * static_cast<int64_t>(p.Fp);
        e = run_tiles<kDw>(k, dp, a.C, p.pieces, static_cast<Tile>(p.tile), whole && aligned(k.x), s);
        if (e != hipSuccess) return e;
    }
    if (!added) return e;
    SumArgs t{};
    const int64_t n = static_cast<int64_t>(a.F) * a.C, fp = p.Fp;
    if (dx && x_part) add_sum(t, x_part, a.rows * a.C, a.rows * a.C, p.x_pieces, a.dx);
    if (weights && w_part) {
        add_sum(t, w_part, 2 * n, n, p.pieces, a.dwg);
        add_sum(t, w_part + n, 2 * n, n, p.pieces, a.dwu);
    }
    if (sums) {
        add_sum(t, sums, 2 * fp, a.F, summed, a.dbg);
        add_sum(t, sums + fp, 2 * fp, a.F, summed, a.dbu);
    }
    events.next(true);
    return launch_sums(t, kType, s);
}

}  // namespace
}  // namespace convmi
