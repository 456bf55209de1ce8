// Gated feed-forward layer in fp32, on the fp32 matrix instruction: the same
// products as in bf16 (see gated.hip), with operands of any length and
// alignment staged through registers into LDS rows of one contraction index.
#include "gated.hpp"

#include <algorithm>

namespace convmi {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
enum Mode { kFwd, kAgain, kDx, kDw };

constexpr int kThreads = 256;
constexpr int kBK = 16;

// 2 x 2 waves, each TP x 2 tiles of 32x32.
template <int TP>
struct Shape {
    static constexpr int BM = 64 * TP, BN = 128, kPitchP = BM % 64 == 32 ? BM : BM + 32, kPitchQ = BN + 32;
};

struct Product {
    const float *x, *wg, *wu, *bg, *bu, *dh, *d;
    float *h, *out, *out2, *d_out, *saved, *sums, *part;
    int64_t rows, per;
    int C, F, Fp, act;
    int p_tiles, q_tiles;
};

// Eight consecutive values from p, n of them there.
__device__ __forceinline__ void load8(const float* p, int64_t n, float* v)
{
    if (n >= 8) {
        const uint4 a = load16_any(p), b = load16_any(p + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.f;
    }
}

template <int TP, int MODE>
__global__ __launch_bounds__(kThreads) void gated_f32_kernel(Product a)
{
    typedef Shape<TP> S;
    constexpr bool kGated = MODE == kFwd || MODE == kAgain;
    constexpr bool kPRows = MODE != kDw, kQRows = kGated;
    constexpr int kQTile = kGated ? S::BN / 2 : S::BN;
    constexpr int kPN = S::BM * kBK / 8 / kThreads > 0 ? S::BM * kBK / 8 / kThreads : 1, kQN = S::BN * kBK / 8 / kThreads;
    __shared__ __align__(16) float ps[2][kBK][S::kPitchP];
    __shared__ __align__(16) float qs[2][kBK][S::kPitchQ];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wp = wave >> 1, wq = wave & 1, col = lane & 31, q = lane >> 5;
    const int tiles = a.p_tiles * a.q_tiles, piece = blockIdx.x / tiles, t = blockIdx.x - piece * tiles;
    const int pt = t % a.p_tiles, qt = t / a.p_tiles;
    const int64_t p0 = static_cast<int64_t>(pt) * S::BM, q0 = static_cast<int64_t>(qt) * kQTile;
    const int64_t m0 = MODE == kDw ? piece * a.per : 0;
    const int64_t K = kGated ? a.C : MODE == kDx ? 2 * static_cast<int64_t>(a.Fp) : min(a.per, a.rows - m0);
    const int64_t p_rows = MODE == kDw ? 2 * static_cast<int64_t>(a.Fp) : a.rows;

    // A thread's eight values of each operand: of one row (along K), or of
    // one contraction index (along the columns).
    float pv[kPN][8], qv[kQN][8];
    const bool p_on = S::BM * kBK / 8 >= kThreads || tid < S::BM * kBK / 8;
    auto load = [&](int64_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kPN; ++i) {
            const int idx = i * kThreads + tid;
            int64_t n = 0;
            const float* src = a.x;
            if (kPRows) {
                const int64_t r = p0 + idx / (kBK / 8), k = k0 + idx % (kBK / 8) * 8;
                const int64_t ld = kGated ? a.C : 2 * static_cast<int64_t>(a.Fp);
                if (r < p_rows) n = K - k, src = (kGated ? a.x : a.d) + r * ld + k;
            } else {
                const int64_t k = k0 + idx / (S::BM / 8), c = p0 + idx % (S::BM / 8) * 8;
                if (k < K) n = p_rows - c, src = a.d + (m0 + k) * 2 * a.Fp + c;
            }
            if (p_on) load8(src, n, pv[i]);
        }
#pragma unroll
        for (int i = 0; i < kQN; ++i) {
            const int idx = i * kThreads + tid;
            int64_t n = 0;
            const float* src = a.x;
            if (kQRows) {
                const int r = idx / (kBK / 8);
                const int64_t k = k0 + idx % (kBK / 8) * 8, f = q0 + (r >> 6) * 32 + (r & 31);
                if (f < a.F) n = K - k, src = (r & 32 ? a.wu : a.wg) + f * a.C + k;
            } else {
                int64_t k = k0 + idx / (S::BN / 8), c = q0 + idx % (S::BN / 8) * 8;
                if (MODE == kDx) {
                    const bool up = k >= a.Fp;
                    k -= up ? a.Fp : 0;
                    if (k < a.F) n = a.C - c, src = (up ? a.wu : a.wg) + k * a.C + c;
                } else if (k < K) {
                    n = a.C - c, src = a.x + (m0 + k) * a.C + c;
                }
            }
            load8(src, n, qv[i]);
        }
    };
    auto put = [&](int st) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kPN; ++i) {
            const int idx = i * kThreads + tid;
            if (!p_on) break;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (kPRows) ps[st][idx % (kBK / 8) * 8 + e][idx / (kBK / 8)] = pv[i][e];
                else ps[st][idx / (S::BM / 8)][idx % (S::BM / 8) * 8 + e] = pv[i][e];
        }
#pragma unroll
        for (int i = 0; i < kQN; ++i) {
            const int idx = i * kThreads + tid;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (kQRows) qs[st][idx % (kBK / 8) * 8 + e][idx / (kBK / 8)] = qv[i][e];
                else qs[st][idx / (S::BN / 8)][idx % (S::BN / 8) * 8 + e] = qv[i][e];
        }
    };

    f32x16 acc[2][TP];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < TP; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

    int st = 0;
    if (K > 0) {
        load(0);
        put(0);
    }
    for (int64_t k0 = 0; k0 < K; k0 += kBK, st ^= 1) {
        __syncthreads();
        const bool more = k0 + kBK < K;
        if (more) load(k0 + kBK);
#pragma unroll
        for (int kk = 0; kk < kBK; kk += 2) {
            float pf[TP], qf[2];
#pragma unroll
            for (int j = 0; j < TP; ++j) pf[j] = ps[st][kk + q][(wp * TP + j) * 32 + col];
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[i] = qs[st][kk + q][(wq * 2 + i) * 32 + col];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < TP; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(qf[i], pf[j], acc[i][j], 0, 0, 0);
        }
        if (more) put(st ^ 1);  // the stage read before the last barrier
    }

    // A lane holds columns 8v + 4q + {0..3} of a q tile and p row `col`.
    if constexpr (kGated) {
        with_act(a.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t f = q0 + wq * 32 + 8 * v + 4 * q + e;
                const float bg = a.bg && f < a.F ? a.bg[f] : 0.f, bu = a.bu && f < a.F ? a.bu[f] : 0.f;
                float sg = 0.f, su = 0.f;
#pragma unroll
                for (int j = 0; j < TP; ++j) {
                    const int64_t r = p0 + (wp * TP + j) * 32 + col;
                    const float g = acc[0][j][4 * v + e] + bg, u = acc[1][j][4 * v + e] + bu;
                    if (r >= a.rows || f >= a.F) continue;
                    if (MODE == kFwd) {
                        if (a.saved) a.saved[r * 2 * a.F + f] = g, a.saved[r * 2 * a.F + a.F + f] = u;
                        a.h[r * a.F + f] = act_value<kind()>(g) * u;
                    } else {
                        const ActPair p = act_pair<kind()>(g);
                        const float dh = a.dh[r * a.F + f], dg = dh * u * p.d, du = dh * p.v;
                        a.d_out[r * 2 * a.Fp + f] = dg;
                        a.d_out[r * 2 * a.Fp + a.Fp + f] = du;
                        sg += dg;
                        su += du;
                    }
                }
                if (MODE == kAgain) {
                    if (a.sums) {
                        for (int s = 1; s < 32; s <<= 1) sg += __shfl_xor(sg, s), su += __shfl_xor(su, s);
                        float* row = a.sums + static_cast<int64_t>(pt * 2 + wp) * 2 * a.Fp;
                        if (col == 0 && f < a.F) row[f] = sg, row[a.Fp + f] = su;
                    }
                    if (f >= a.F && f < a.Fp)  // the columns past F are operands of the products: zero
#pragma unroll
                        for (int j = 0; j < TP; ++j) {
                            const int64_t r = p0 + (wp * TP + j) * 32 + col;
                            if (r < a.rows) a.d_out[r * 2 * a.Fp + f] = a.d_out[r * 2 * a.Fp + a.Fp + f] = 0.f;
                        }
                }
            }
        });
    } else {
#pragma unroll
        for (int j = 0; j < TP; ++j) {
            const int64_t r = p0 + (wp * TP + j) * 32 + col;
            float* row;
            if (MODE == kDx) {
                row = r < a.rows ? a.out + r * a.C : nullptr;
            } else {
                const int half = r >= a.Fp;
                const int64_t f = r - (half ? a.Fp : 0);
                float* w = half ? a.out2 : a.out;
                row = f >= a.F || r >= 2 * static_cast<int64_t>(a.Fp) ? nullptr
                      : a.part ? a.part + ((static_cast<int64_t>(piece) * 2 + half) * a.F + f) * a.C
                               : w ? w + f * a.C : nullptr;
            }
            if (!row) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int64_t c = q0 + (wq * 2 + i) * 32 + 8 * (v >> 2) + 4 * q + (v & 3);
                    if (c < a.C) row[c] = acc[i][j][v];
                }
        }
    }
}

int64_t tiles(int64_t n, int t) { return (n + t - 1) / t; }

template <int MODE>
hipError_t run(Product& k, int64_t p, int64_t q, int pieces, bool big, hipStream_t s)
{
    k.p_tiles = static_cast<int>(tiles(p, big ? Shape<2>::BM : Shape<1>::BM));
    k.q_tiles = static_cast<int>(tiles(q, 128));
    const int64_t blocks = static_cast<int64_t>(k.p_tiles) * k.q_tiles * pieces;
    if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    return launch(big ? gated_f32_kernel<2, MODE> : gated_f32_kernel<1, MODE>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, k);
}

// 128-row tiles once they give every CU two workgroups.
bool use_big(int64_t p, int64_t q) { return tiles(p, 128) * tiles(q, 128) >= 2 * device_cu_count(); }

Product product(const GatedArgs& a)
{
    Product k{};
    k.x = static_cast<const float*>(a.x);
    k.wg = static_cast<const float*>(a.wg);
    k.wu = static_cast<const float*>(a.wu);
    k.bg = static_cast<const float*>(a.bg);
    k.bu = static_cast<const float*>(a.bu);
    k.dh = static_cast<const float*>(a.dh);
    k.rows = a.rows;
    k.C = a.C;
    k.F = a.F;
    k.act = a.act;
    return k;
}

}  // namespace

GatedPlan gated_plan_f32(int64_t rows, int C, int F)
{
    GatedPlan p{};
    p.Fp = (F + 15) / 16 * 16;
    const bool big = use_big(2 * static_cast<int64_t>(p.Fp), C);
    const int64_t t = tiles(2 * static_cast<int64_t>(p.Fp), big ? 128 : 64) * tiles(C, 128);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(3 * device_cu_count() / t, rows / 128));
    p.per = std::max<int64_t>(kBK, (tiles(rows, static_cast<int>(want)) + kBK - 1) / kBK * kBK);
    p.pieces = static_cast<int>(std::max<int64_t>(1, (rows + p.per - 1) / p.per));
    int64_t chunk;
    p.sum_rows = static_cast<int>(std::max<int64_t>(gated_kept_chunks(rows, p.Fp, &chunk), tiles(rows, 64) * 2));
    p.d_bytes = round256(static_cast<size_t>(rows) * 2 * p.Fp * 4);
    p.sum_bytes = round256(static_cast<size_t>(p.sum_rows) * 2 * p.Fp * 4);
    p.part_bytes = p.pieces > 1 ? round256(static_cast<size_t>(p.pieces) * 2 * F * C * 4) : 0;
    return p;
}

hipError_t gated_fwd_f32(const GatedArgs& a, hipStream_t s)
{
    Product k = product(a);
    k.h = static_cast<float*>(a.h);
    k.saved = a.saved;
    const int64_t q = 2 * static_cast<int64_t>(a.F);
    return run<kFwd>(k, a.rows, q, 1, use_big(a.rows, q), s);
}

hipError_t gated_bwd_f32(const GatedArgs& a, hipStream_t s)
{
    const GatedPlan p = gated_plan_f32(a.rows, a.C, a.F);
    char* ws = static_cast<char*>(a.workspace);
    float* d = reinterpret_cast<float*>(ws);
    float* sums = a.dbg || a.dbu ? reinterpret_cast<float*>(ws + p.d_bytes) : nullptr;
    float* part = reinterpret_cast<float*>(ws + p.d_bytes + p.sum_bytes);
    const ArmedEvents armed = armed_events();
    armed_events() = ArmedEvents{armed.start, nullptr};
    hipError_t e = hipSuccess;
    int sum_rows = 0;
    Product k = product(a);
    k.Fp = p.Fp;
    if (a.rows > 0) {
        if (a.saved) {
            int64_t chunk;
            sum_rows = gated_kept_chunks(a.rows, p.Fp, &chunk);
            e = launch_gated_kept(a, d, sums, p.Fp, sum_rows, chunk, 0, s);
        } else {
            k.d_out = d;
            k.sums = sums;
            const int64_t q = 2 * static_cast<int64_t>(a.F);
            const bool big = use_big(a.rows, q);
            sum_rows = static_cast<int>(tiles(a.rows, big ? 128 : 64)) * 2;
            e = run<kAgain>(k, a.rows, q, 1, big, s);
        }
        armed_events() = ArmedEvents{nullptr, nullptr};
        if (e != hipSuccess) return e;
        k.d = d;
        if (a.dx) {
            k.out = static_cast<float*>(a.dx);
            e = run<kDx>(k, a.rows, a.C, 1, use_big(a.rows, a.C), s);
            if (e != hipSuccess) return e;
        }
    }
    if (sums) {
        e = launch_gated_bias_sums(a, sums, sum_rows, p.Fp, 0, s);
        if (e != hipSuccess) return e;
    }
    if (a.dwg || a.dwu) {
        k.d = d;
        k.out = static_cast<float*>(a.dwg);
        k.out2 = static_cast<float*>(a.dwu);
        k.part = p.pieces > 1 ? part : nullptr;
        k.per = p.per;
        if (p.pieces == 1) armed_events() = ArmedEvents{nullptr, armed.stop};
        const int64_t rows2 = 2 * static_cast<int64_t>(p.Fp);
        e = run<kDw>(k, rows2, a.C, p.pieces, use_big(rows2, a.C), s);
        armed_events() = ArmedEvents{nullptr, p.pieces > 1 ? armed.stop : nullptr};
        if (e == hipSuccess && p.pieces > 1) e = launch_gated_weight_sums(a, part, p.pieces, 0, s);
    }
    armed_events() = ArmedEvents{nullptr, nullptr};
    return e;
}

}  // namespace convmi
