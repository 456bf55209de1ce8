// C ABI of the operators along a sequence: argument checks and launches of the
// short causal convolution and the selective scan.  Every check runs on the
// host before anything is launched.
#include "checks.hpp"

using namespace convmi::checks;
using convmi::fail;

namespace {

constexpr long long kMaxStride = (1 << 24) - 1;  // elements from one row to the next

size_t size_of(int dtype) { return dtype == CONV_F32 ? 4 : 2; }

// A tensor of a call: its first byte, its bytes, and whether the call writes it.
struct Part {
    const void* at;
    int64_t count;  // elements
    size_t size;    // of an element
    bool written;
};
Part dense(const void* p, int64_t n, size_t size) { return {p, p ? n : 0, size, false}; }
Part out(const void* p, int64_t n, size_t size) { return {p, p ? n : 0, size, true}; }
Part strided(const void* p, int64_t rows, int64_t stride, int64_t width, size_t size)
{
    return {p, p && rows > 0 ? (rows - 1) * stride + width : 0, size, false};
}

int check_parts(const char* op, std::initializer_list<Part> parts)
{
    Span s[32];
    int m = 0;
    for (const Part& p : parts) {
        if (p.count > 0 && off(p.at, p.size)) return fail(CONV_ERR_INVALID_ARG, "%s: a tensor is not aligned to its %zu-byte elements", op, p.size);
        if (p.count <= 0) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p.at);
        s[m++] = Span{at, at + static_cast<size_t>(p.count) * p.size, p.written};
    }
    if (!spans_apart(s, m)) return fail(CONV_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", op);
    return CONV_OK;
}

int check_stride(const char* op, const char* name, long long stride, long long width)
{
    if (stride < width || stride > kMaxStride)
        return fail(stride < width ? CONV_ERR_INVALID_ARG : CONV_ERR_OVERFLOW, "%s: %s_stride must be at least %lld and below 2^24 (got %lld)", op, name, width,
                    stride);
    return CONV_OK;
}

int check_sequences(const char* op, long long rows, int seqs, bool packed)
{
    if (seqs < 0 || (seqs == 0 && rows > 0))
        return fail(CONV_ERR_INVALID_ARG, "%s: seqs must be >= 0, and >= 1 with rows (got %d for %lld)", op, seqs, rows);
    if (!packed && seqs > 0 && rows % seqs != 0)
        return fail(CONV_ERR_INVALID_ARG, "%s: %d sequences do not divide %lld rows (and there are no starts)", op, seqs, rows);
    return CONV_OK;
}

int check_causal(const char* op, const convmi::CausalArgs& a, long long rows, int C, int K, long long x_stride, int act, int dtype)
{
    int rc = check_dtype(op, dtype);
    if (!rc) rc = check_act(op, act);
    if (!rc) rc = check_sizes(op, rows, C, "C");
    if (!rc) rc = check_stride(op, "x", x_stride, C);
    if (rc) return rc;
    if (K < 2 || K > convmi::kCausalTaps) return fail(CONV_ERR_INVALID_ARG, "%s: K must be 2 to %d, got %d", op, convmi::kCausalTaps, K);
    if (rows > 0 && (!a.x || !a.w)) return fail(CONV_ERR_INVALID_ARG, "%s: x and w must not be NULL", op);
    return CONV_OK;
}

int check_scan_sizes(const char* op, long long rows, int channels, int N, int groups)
{
    if (int rc = check_sizes(op, rows, channels, "channels")) return rc;
    if (N < 1 || N > convmi::kScanStates) return fail(CONV_ERR_INVALID_ARG, "%s: N must be 1 to %d, got %d", op, convmi::kScanStates, N);
    if (groups < 1 || channels % groups != 0 || groups > 65535)
        return fail(CONV_ERR_INVALID_ARG, "%s: groups must divide the %d channels (and be below 65536), got %d", op, channels, groups);
    return CONV_OK;
}

int check_scan(const char* op, const convmi::ScanArgs& a, int N, int dtype)
{
    int rc = check_dtype(op, dtype);
    if (!rc) rc = check_act(op, a.act);
    if (!rc) rc = check_scan_sizes(op, a.rows, a.channels, N, a.groups);
    const long long states = static_cast<long long>(a.groups) * N;
    if (!rc) rc = check_stride(op, "x", a.xs, a.channels);
    if (!rc) rc = check_stride(op, "delta", a.ds, a.channels);
    if (!rc && a.z) rc = check_stride(op, "z", a.zs, a.channels);
    if (!rc) rc = check_stride(op, "B", a.bs, states);
    if (!rc) rc = check_stride(op, "C", a.cs, states);
    if (rc) return rc;
    if (!a.A || (a.rows > 0 && (!a.x || !a.delta || !a.B || !a.C)))
        return fail(CONV_ERR_INVALID_ARG, "%s: x, delta, A, B and C must not be NULL", op);
    return CONV_OK;
}

convmi::ScanArgs scan_args(const void* x, const void* delta, const float* A, const void* B, const void* C, const float* D, const void* z,
                           const float* bias, long long rows, int seqs, int channels, int N, int groups, long long xs, long long ds,
                           long long zs, long long bs, long long cs, int softplus, int act, int clear)
{
    convmi::ScanArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = bias;
    a.rows = rows; a.seqs = seqs; a.channels = channels; a.n = N; a.groups = groups;
    a.len = seqs > 0 ? rows / seqs : 0;
    a.per_group = groups > 0 ? channels / groups : 0;
    a.xs = xs; a.ds = ds; a.zs = zs; a.bs = bs; a.cs = cs;
    a.softplus = softplus != 0; a.act = act; a.clear = clear != 0;
    return a;
}

}  // namespace

extern "C" {

int conv_causal_fwd(const void* x, const void* w, const void* bias, const int* starts, const void* initial, void* y, void* last, long long rows,
                    int seqs, int C, int K, long long x_stride, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_causal_fwd";
    convmi::CausalArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.starts = starts; a.initial = initial; a.y = y; a.last = last;
    if (int rc = check_causal(op, a, rows, C, K, x_stride, act, dtype)) return rc;
    if (int rc = check_sequences(op, rows, seqs, starts != nullptr)) return rc;
    if (rows > 0 && !y) return fail(CONV_ERR_INVALID_ARG, "%s: y must not be NULL", op);
    const size_t e = size_of(dtype);
    const int64_t n = static_cast<int64_t>(rows) * C, states = static_cast<int64_t>(seqs) * (K - 1) * C;
    if (int rc = check_parts(op, {strided(x, rows, x_stride, C, e), dense(w, static_cast<int64_t>(C) * K, e), dense(bias, C, e),
                                  dense(starts, seqs + 1LL, 4), dense(initial, states, e), out(y, n, e), out(last, states, e)})) return rc;
    a.rows = rows; a.len = seqs > 0 ? rows / seqs : 0; a.xs = x_stride; a.seqs = seqs; a.C = C; a.K = K; a.act = act; a.clear = clear != 0;
    return launched(convmi::launch_causal_fwd(a, dtype, static_cast<hipStream_t>(stream)), op);
}

int conv_causal_bwd_workspace_size(long long rows, int C, int K, int dtype, size_t* bytes)
{
    static const char* op = "conv_causal_bwd_workspace_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_dtype(op, dtype)) return rc;
    if (int rc = check_sizes(op, rows, C, "C")) return rc;
    if (K < 2 || K > convmi::kCausalTaps) return fail(CONV_ERR_INVALID_ARG, "%s: K must be 2 to %d, got %d", op, convmi::kCausalTaps, K);
    *bytes = convmi::causal_bwd_workspace(rows, C, K);
    return CONV_OK;
}

int conv_causal_bwd(const void* dy, const void* dlast, const void* x, const void* w, const void* bias, const int* starts, const void* initial,
                    void* dx, void* dw, void* dbias, void* dinitial, void* workspace, size_t workspace_bytes, long long rows, int seqs, int C,
                    int K, long long x_stride, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_causal_bwd";
    convmi::CausalArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.starts = starts; a.initial = initial; a.dy = dy; a.dlast = dlast; a.dx = dx; a.dinitial = dinitial;
    if (int rc = check_causal(op, a, rows, C, K, x_stride, act, dtype)) return rc;
    if (int rc = check_sequences(op, rows, seqs, starts != nullptr)) return rc;
    if (rows > 0 && !dy) return fail(CONV_ERR_INVALID_ARG, "%s: dy must not be NULL", op);
    const size_t e = size_of(dtype), need = convmi::causal_bwd_workspace(rows, C, K);
    if (int rc = check_workspace(op, workspace, workspace_bytes, need)) return rc;
    const int64_t n = static_cast<int64_t>(rows) * C, states = static_cast<int64_t>(seqs) * (K - 1) * C, wn = static_cast<int64_t>(C) * K;
    if (int rc = check_parts(op, {dense(dy, n, e), dense(dlast, states, e), strided(x, rows, x_stride, C, e), dense(w, wn, e), dense(bias, C, e),
                                  dense(starts, seqs + 1LL, 4), dense(initial, states, e), out(dx, n, e), out(dw, wn, e), out(dbias, C, e),
                                  out(dinitial, states, e), out(workspace, static_cast<int64_t>(need), 1)})) return rc;
    a.rows = rows; a.len = seqs > 0 ? rows / seqs : 0; a.xs = x_stride; a.seqs = seqs; a.C = C; a.K = K; a.act = act; a.clear = clear != 0;
    return launched(convmi::launch_causal_bwd(a, dw, dbias, dtype, workspace, static_cast<hipStream_t>(stream)), op);
}

int conv_causal_step(const void* x, const void* w, const void* bias, void* state, const int* slots, void* y, long long rows, int count, int C,
                     int K, long long x_stride, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_causal_step";
    convmi::CausalArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.slots = slots; a.y = y;
    if (int rc = check_causal(op, a, rows, C, K, x_stride, act, dtype)) return rc;
    if (count < 0 || (!slots && rows > count)) return fail(CONV_ERR_INVALID_ARG, "%s: %d states for %lld rows without slots", op, count, rows);
    if (rows > 0 && (!y || (!state && count > 0))) return fail(CONV_ERR_INVALID_ARG, "%s: state and y must not be NULL", op);
    const size_t e = size_of(dtype);
    if (int rc = check_parts(op, {strided(x, rows, x_stride, C, e), dense(w, static_cast<int64_t>(C) * K, e), dense(bias, C, e), dense(slots, rows, 4),
                                  out(state, static_cast<int64_t>(count) * (K - 1) * C, e), out(y, static_cast<int64_t>(rows) * C, e)})) return rc;
    a.rows = rows; a.xs = x_stride; a.C = C; a.K = K; a.act = act; a.clear = clear != 0;
    return launched(convmi::launch_causal_step(a, count, dtype, static_cast<hipStream_t>(stream)), op);
}

int conv_scan_saved_size(long long rows, int channels, int N, size_t* bytes)
{
    static const char* op = "conv_scan_saved_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_scan_sizes(op, rows, channels, N, 1)) return rc;
    *bytes = convmi::scan_saved(rows, channels, N);
    return CONV_OK;
}

static int scan_workspace(const char* op, bool gradient, long long rows, int seqs, int channels, int N, int groups, int packed, int saved, size_t* bytes)
{
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_scan_sizes(op, rows, channels, N, groups)) return rc;
    if (int rc = check_sequences(op, rows, seqs, packed != 0)) return rc;
    const convmi::ScanArgs a = scan_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, rows, seqs, channels, N, groups, 0, 0, 0,
                                         0, 0, 0, 0, 0);
    *bytes = gradient ? convmi::scan_bwd_workspace(a, packed != 0, saved != 0) : convmi::scan_fwd_workspace(a, packed != 0);
    return CONV_OK;
}

int conv_scan_fwd_workspace_size(long long rows, int seqs, int channels, int N, int groups, int packed, size_t* bytes)
{
    return scan_workspace("conv_scan_fwd_workspace_size", false, rows, seqs, channels, N, groups, packed, 0, bytes);
}

int conv_scan_bwd_workspace_size(long long rows, int seqs, int channels, int N, int groups, int packed, int saved, size_t* bytes)
{
    return scan_workspace("conv_scan_bwd_workspace_size", true, rows, seqs, channels, N, groups, packed, saved, bytes);
}

int conv_scan_fwd(const void* x, const void* delta, const float* A, const void* B, const void* C, const float* D, const void* z,
                  const float* delta_bias, const int* starts, const float* initial, void* y, float* last, float* saved, void* workspace,
                  size_t workspace_bytes, long long rows, int seqs, int channels, int N, int groups, long long x_stride, long long delta_stride,
                  long long z_stride, long long B_stride, long long C_stride, int softplus, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_scan_fwd";
    convmi::ScanArgs a = scan_args(x, delta, A, B, C, D, z, delta_bias, rows, seqs, channels, N, groups, x_stride, delta_stride, z_stride, B_stride,
                                   C_stride, softplus, act, clear);
    a.starts = starts; a.initial = initial; a.y = y; a.last = last; a.saved = saved;
    if (int rc = check_scan(op, a, N, dtype)) return rc;
    if (int rc = check_sequences(op, rows, seqs, starts != nullptr)) return rc;
    if (rows > 0 && !y) return fail(CONV_ERR_INVALID_ARG, "%s: y must not be NULL", op);
    const size_t need = convmi::scan_fwd_workspace(a, starts != nullptr);
    if (int rc = check_workspace(op, workspace, workspace_bytes, need)) return rc;
    const size_t e = size_of(dtype);
    const int64_t n = static_cast<int64_t>(rows) * channels, one = static_cast<int64_t>(channels) * N, states = seqs * one, bc = static_cast<int64_t>(groups) * N;
    if (int rc = check_parts(op, {strided(x, rows, x_stride, channels, e), strided(delta, rows, delta_stride, channels, e), strided(z, rows, z_stride, channels, e),
                                  strided(B, rows, B_stride, bc, e), strided(C, rows, C_stride, bc, e), dense(A, one, 4), dense(D, channels, 4),
                                  dense(delta_bias, channels, 4), dense(starts, seqs + 1LL, 4), dense(initial, states, 4), out(y, n, e),
                                  out(last, states, 4), out(saved, static_cast<int64_t>(convmi::scan_saved(rows, channels, N) / 4), 4),
                                  out(workspace, static_cast<int64_t>(need), 1)})) return rc;
    return launched(convmi::launch_scan_fwd(a, dtype, workspace, static_cast<hipStream_t>(stream)), op);
}

int conv_scan_bwd(const void* dy, const float* dlast, const void* x, const void* delta, const float* A, const void* B, const void* C, const float* D,
                  const void* z, const float* delta_bias, const int* starts, const float* initial, const float* saved, void* dx, void* ddelta, float* dA,
                  void* dB, void* dC, float* dD, void* dz, float* ddelta_bias, float* dinitial, void* workspace, size_t workspace_bytes, long long rows,
                  int seqs, int channels, int N, int groups, long long x_stride, long long delta_stride, long long z_stride, long long B_stride,
                  long long C_stride, int softplus, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_scan_bwd";
    convmi::ScanArgs a = scan_args(x, delta, A, B, C, D, z, delta_bias, rows, seqs, channels, N, groups, x_stride, delta_stride, z_stride, B_stride,
                                   C_stride, softplus, act, clear);
    a.starts = starts; a.initial = initial; a.saved = const_cast<float*>(saved); a.dy = dy; a.dlast = dlast;
    a.dx = dx; a.ddelta = ddelta; a.dB = dB; a.dC = dC; a.dz = dz; a.dinitial = dinitial;
    if (int rc = check_scan(op, a, N, dtype)) return rc;
    if (int rc = check_sequences(op, rows, seqs, starts != nullptr)) return rc;
    if (rows > 0 && !dy) return fail(CONV_ERR_INVALID_ARG, "%s: dy must not be NULL", op);
    if (dz && !z) return fail(CONV_ERR_INVALID_ARG, "%s: dz needs z", op);
    const size_t need = convmi::scan_bwd_workspace(a, starts != nullptr, saved != nullptr);
    if (int rc = check_workspace(op, workspace, workspace_bytes, need)) return rc;
    const size_t e = size_of(dtype);
    const int64_t n = static_cast<int64_t>(rows) * channels, one = static_cast<int64_t>(channels) * N, states = seqs * one, bc = static_cast<int64_t>(groups) * N;
    if (int rc = check_parts(op, {dense(dy, n, e), dense(dlast, states, 4), strided(x, rows, x_stride, channels, e), strided(delta, rows, delta_stride, channels, e),
                                  strided(z, rows, z_stride, channels, e), strided(B, rows, B_stride, bc, e), strided(C, rows, C_stride, bc, e), dense(A, one, 4),
                                  dense(D, channels, 4), dense(delta_bias, channels, 4), dense(starts, seqs + 1LL, 4), dense(initial, states, 4),
                                  dense(saved, static_cast<int64_t>(convmi::scan_saved(rows, channels, N) / 4), 4), out(dx, n, e), out(ddelta, n, e), out(dz, n, e),
                                  out(dA, one, 4), out(dB, rows * bc, e), out(dC, rows * bc, e), out(dD, channels, 4), out(ddelta_bias, channels, 4),
                                  out(dinitial, states, 4), out(workspace, static_cast<int64_t>(need), 1)})) return rc;
    convmi::ScanGrads g{dA, dD, ddelta_bias};
    return launched(convmi::launch_scan_bwd(a, g, dtype, workspace, static_cast<hipStream_t>(stream)), op);
}

int conv_scan_step(const void* x, const void* delta, const float* A, const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                   float* state, const int* slots, void* y, long long rows, int count, int channels, int N, int groups, long long x_stride,
                   long long delta_stride, long long z_stride, long long B_stride, long long C_stride, int softplus, int act, int clear, int dtype, void* stream)
{
    static const char* op = "conv_scan_step";
    convmi::ScanArgs a = scan_args(x, delta, A, B, C, D, z, delta_bias, rows, 0, channels, N, groups, x_stride, delta_stride, z_stride, B_stride, C_stride,
                                   softplus, act, clear);
    a.slots = slots; a.y = y;
    if (int rc = check_scan(op, a, N, dtype)) return rc;
    if (count < 0 || (!slots && rows > count)) return fail(CONV_ERR_INVALID_ARG, "%s: %d states for %lld rows without slots", op, count, rows);
    if (rows > 0 && (!y || (!state && count > 0))) return fail(CONV_ERR_INVALID_ARG, "%s: state and y must not be NULL", op);
    const size_t e = size_of(dtype);
    const int64_t one = static_cast<int64_t>(channels) * N, bc = static_cast<int64_t>(groups) * N;
    if (int rc = check_parts(op, {strided(x, rows, x_stride, channels, e), strided(delta, rows, delta_stride, channels, e), strided(z, rows, z_stride, channels, e),
                                  strided(B, rows, B_stride, bc, e), strided(C, rows, C_stride, bc, e), dense(A, one, 4), dense(D, channels, 4),
                                  dense(delta_bias, channels, 4), dense(slots, rows, 4), out(state, count * one, 4),
                                  out(y, static_cast<int64_t>(rows) * channels, e)})) return rc;
    return launched(convmi::launch_scan_step(a, state, count, dtype, static_cast<hipStream_t>(stream)), op);
}

}  // extern "C"
