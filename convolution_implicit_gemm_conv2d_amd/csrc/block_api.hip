// C ABI of the operators around a convolution: argument checks and launches of
// the gated feed-forward layer, the block norms and gradient clipping.  Every
// check runs on the host before anything is launched.
#include "checks.hpp"

#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

using namespace convmi::checks;
using convmi::fail;

static_assert(convmi::kActs == CONV_ACT_TANH + 1, "the activations of the header");

namespace {

int check_gated(const char* op, long long rows, int C, int F, int act, int dtype)
{
    int rc = check_dtype(op, dtype);
    if (!rc) rc = check_act(op, act);
    if (!rc) rc = check_sizes(op, rows, C, "C");
    if (!rc) rc = check_sizes(op, rows, F, "F");
    return rc;
}

int check_norm(const char* op, const convmi::NormArgs& a, long long rows, int C, long long gate_rows, int dtype)
{
    int rc = check_dtype(op, dtype);
    if (!rc) rc = check_act(op, a.act);
    if (!rc) rc = check_sizes(op, rows, C, "C");
    if (rc) return rc;
    if (a.post < CONV_NORM_NONE || a.post > CONV_NORM_LAYER || a.pre < CONV_NORM_NONE || a.pre > CONV_NORM_LAYER)
        return fail(CONV_ERR_INVALID_ARG, "%s: post and pre must be conv_norm_t values", op);
    if (!(a.eps > 0.f) || !std::isfinite(a.eps))
        return fail(CONV_ERR_INVALID_ARG, "%s: eps must be positive and finite", op);
    if (!a.x && rows > 0) return fail(CONV_ERR_INVALID_ARG, "%s: x must not be NULL", op);
    if (!a.f && rows > 0 && (a.z || a.s || a.post != CONV_NORM_NONE))
        return fail(CONV_ERR_INVALID_ARG, "%s: a gate, a scale or a post norm needs a branch", op);
    if (a.z && (gate_rows < 1 || rows % gate_rows != 0))
        return fail(CONV_ERR_INVALID_ARG, "%s: gate_rows must be >= 1 and divide rows (got %lld for %lld)", op, gate_rows, rows);
    if ((a.post_w && a.post == CONV_NORM_NONE) || (a.pre_w && a.pre == CONV_NORM_NONE) ||
        (a.post_b && a.post != CONV_NORM_LAYER) || (a.pre_b && a.pre != CONV_NORM_LAYER))
        return fail(CONV_ERR_INVALID_ARG, "%s: a weight needs its norm, a bias its layer norm", op);
    return check_aligned(op, {a.dy, a.da, a.x, a.f, a.z, a.s, a.post_w, a.post_b, a.pre_w, a.pre_b, a.y, a.a, a.dx, a.df,
                              a.dz, a.ds, a.dpost_w, a.dpost_b, a.dpre_w, a.dpre_b}, dtype == CONV_F32 ? 4 : 2);
}

// Clipping writes a list's outputs in any order, many workgroups at a time: none
// may overlap another output, or a gradient but the one it replaces.  A list of
// 600 tensors takes 15 us.
int check_apart(const char* op, const void* const* grads, void* const* outs, const size_t* counts, const int* dtypes, int n)
{
    constexpr int kHere = 512;
    Span here[kHere];
    std::unique_ptr<Span[]> more;
    Span* s = here;
    if (2 * static_cast<int64_t>(n) > kHere) {
        more.reset(new (std::nothrow) Span[2 * static_cast<size_t>(n)]);
        if (!more) return fail(CONV_ERR_HIP, "%s: no host memory to check %d tensors", op, n);
        s = more.get();
    }
    int m = 0;
    for (int i = 0; i < n; ++i) {
        if (counts[i] == 0) continue;
        const size_t bytes = counts[i] * (dtypes[i] == CONV_F32 ? 4 : 2);
        const uintptr_t to = reinterpret_cast<uintptr_t>(outs[i]), from = reinterpret_cast<uintptr_t>(grads[i]);
        s[m++] = Span{to, to + bytes, true};
        if (from != to) s[m++] = Span{from, from + bytes, false};
    }
    if (!spans_apart(s, m)) return fail(CONV_ERR_INVALID_ARG, "%s: an output overlaps another output or another gradient", op);
    return CONV_OK;
}

int check_list(const char* op, const void* const* grads, void* const* outs, bool clip, const size_t* counts,
               const int* dtypes, int n, const void* workspace, size_t bytes)
{
    if (n < 0) return fail(CONV_ERR_INVALID_ARG, "%s: n must be >= 0, got %d", op, n);
    if (n > 0 && (!grads || !counts || !dtypes || (clip && !outs)))
        return fail(CONV_ERR_INVALID_ARG, "%s: an array is NULL", op);
    for (int i = 0; i < n; ++i) {
        if (int rc = check_dtype(op, dtypes[i])) return rc;
        if (counts[i] == 0) continue;
        if (counts[i] >> 46) return fail(CONV_ERR_OVERFLOW, "%s: tensor %d has 2^46 elements or more", op, i);
        if (!grads[i] || (clip && !outs[i])) return fail(CONV_ERR_INVALID_ARG, "%s: tensor %d is NULL", op, i);
        const size_t align = dtypes[i] == CONV_F32 ? 4 : 2;
        if (off(grads[i], align) || (clip && off(outs[i], align)))
            return fail(CONV_ERR_INVALID_ARG, "%s: tensor %d is not aligned to its %zu-byte elements", op, i, align);
    }
    if (clip)
        if (int rc = check_apart(op, grads, outs, counts, dtypes, n)) return rc;
    return check_workspace(op, workspace, bytes, convmi::clip_workspace(n));
}

}  // namespace

extern "C" {

int conv_block_norm_fwd(const void* x, const void* branch, const void* gate, const void* scale, const void* post_w,
                        const void* post_b, const void* pre_w, const void* pre_b, void* y, void* a, long long rows, int C,
                        long long gate_rows, int post, int pre, int act, float eps, int dtype, void* stream)
{
    static const char* op = "conv_block_norm_fwd";
    convmi::NormArgs k{};
    k.x = x; k.f = branch; k.z = gate; k.s = scale;
    k.post_w = post_w; k.post_b = post_b; k.pre_w = pre_w; k.pre_b = pre_b;
    k.y = y; k.a = a;
    k.rows = rows; k.gate_rows = gate ? gate_rows : 1;
    k.C = C; k.post = post; k.pre = pre; k.act = act; k.eps = eps;
    if (int rc = check_norm(op, k, rows, C, gate_rows, dtype)) return rc;
    if (rows > 0 && !y && !a) return fail(CONV_ERR_INVALID_ARG, "%s: y and a must not both be NULL", op);
    if (a && pre == CONV_NORM_NONE) return fail(CONV_ERR_INVALID_ARG, "%s: a needs a pre norm", op);
    return launched(convmi::launch_norm_fwd(k, dtype, static_cast<hipStream_t>(stream)), op);
}

int conv_block_norm_bwd_workspace_size(long long rows, int C, long long gate_rows, size_t* bytes)
{
    static const char* op = "conv_block_norm_bwd_workspace_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_sizes(op, rows, C, "C")) return rc;
    if (gate_rows < 0 || (gate_rows > 0 && rows % gate_rows != 0))
        return fail(CONV_ERR_INVALID_ARG, "%s: gate_rows must divide rows (got %lld for %lld)", op, gate_rows, rows);
    *bytes = convmi::norm_bwd_workspace(rows, C);
    return CONV_OK;
}

int conv_block_norm_bwd(const void* dy, const void* da, const void* x, const void* branch, const void* gate,
                        const void* scale, const void* post_w, const void* post_b, const void* pre_w, const void* pre_b,
                        void* dx, void* dbranch, void* dgate, void* dscale, void* dpost_w, void* dpost_b, void* dpre_w,
                        void* dpre_b, void* workspace, size_t workspace_bytes, long long rows, int C, long long gate_rows,
                        int post, int pre, int act, float eps, int dtype, void* stream)
{
    static const char* op = "conv_block_norm_bwd";
    convmi::NormArgs k{};
    k.dy = dy; k.da = da;
    k.x = x; k.f = branch; k.z = gate; k.s = scale;
    k.post_w = post_w; k.post_b = post_b; k.pre_w = pre_w; k.pre_b = pre_b;
    k.dx = dx; k.df = dbranch; k.dz = dgate; k.ds = dscale;
    k.dpost_w = dpost_w; k.dpost_b = dpost_b; k.dpre_w = dpre_w; k.dpre_b = dpre_b;
    k.part = static_cast<float*>(workspace);
    k.rows = rows; k.gate_rows = gate ? gate_rows : 1;
    k.C = C; k.post = post; k.pre = pre; k.act = act; k.eps = eps;
    if (int rc = check_norm(op, k, rows, C, gate_rows, dtype)) return rc;
    if (rows > 0 && !dy && !da) return fail(CONV_ERR_INVALID_ARG, "%s: dy and da must not both be NULL", op);
    if (da && pre == CONV_NORM_NONE) return fail(CONV_ERR_INVALID_ARG, "%s: da needs a pre norm", op);
    if (rows > 0 && ((dbranch || dscale) && !branch))
        return fail(CONV_ERR_INVALID_ARG, "%s: the gradient of a branch or scale needs a branch", op);
    if (rows > 0 && dgate && !gate) return fail(CONV_ERR_INVALID_ARG, "%s: dgate needs a gate", op);
    if (((dpost_w || dpost_b) && post == CONV_NORM_NONE) || ((dpre_w || dpre_b) && pre == CONV_NORM_NONE) ||
        (dpost_b && post != CONV_NORM_LAYER) || (dpre_b && pre != CONV_NORM_LAYER))
        return fail(CONV_ERR_INVALID_ARG, "%s: a weight gradient needs its norm, a bias gradient its layer norm", op);
    const size_t need = convmi::norm_bwd_workspace(rows, C);
    if (int rc = check_workspace(op, workspace, workspace_bytes, need)) return rc;
    return launched(convmi::launch_norm_bwd(k, dtype, static_cast<hipStream_t>(stream)), op);
}

static int gated_forward(const char* op, const void* x, const void* w_gate, const void* w_up, const void* b_gate, const void* b_up,
                         void* h, float* saved, void* workspace, long long rows, int C, int F, int act, int dtype, void* stream)
{
    if (int rc = check_gated(op, rows, C, F, act, dtype)) return rc;
    if (rows == 0) return CONV_OK;
    if (!x || !w_gate || !w_up || !h)
        return fail(CONV_ERR_INVALID_ARG, "%s: x, w_gate, w_up and h must not be NULL", op);
    if ((b_gate != nullptr) != (b_up != nullptr))
        return fail(CONV_ERR_INVALID_ARG, "%s: b_gate and b_up come together", op);
    if (int rc = check_aligned(op, {x, w_gate, w_up, b_gate, b_up, h}, dtype == CONV_F32 ? 4 : 2)) return rc;
    if (int rc = check_aligned(op, {saved}, 4)) return rc;
    convmi::GatedArgs k{};
    k.x = x; k.wg = w_gate; k.wu = w_up; k.bg = b_gate; k.bu = b_up; k.h = h; k.saved = saved;
    k.workspace = workspace;
    k.rows = rows; k.C = C; k.F = F; k.act = act;
    return launched(convmi::launch_gated_fwd(k, dtype, static_cast<hipStream_t>(stream)), op);
}

int conv_gated_fwd(const void* x, const void* w_gate, const void* w_up, const void* b_gate, const void* b_up, void* h,
                   float* saved, long long rows, int C, int F, int act, int dtype, void* stream)
{
    return gated_forward("conv_gated_fwd", x, w_gate, w_up, b_gate, b_up, h, saved, nullptr, rows, C, F, act, dtype, stream);
}

int conv_gated_fwd_workspace_size(long long rows, int C, int F, int dtype, size_t* bytes)
{
    static const char* op = "conv_gated_fwd_workspace_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_gated(op, rows, C, F, CONV_ACT_NONE, dtype)) return rc;
    *bytes = convmi::gated_fwd_workspace(rows, C, F, dtype);
    return CONV_OK;
}

int conv_gated_fwd_ex(const void* x, const void* w_gate, const void* w_up, const void* b_gate, const void* b_up, void* h,
                      float* saved, void* workspace, size_t workspace_bytes, long long rows, int C, int F, int act, int dtype,
                      void* stream)
{
    static const char* op = "conv_gated_fwd_ex";
    if (int rc = check_gated(op, rows, C, F, act, dtype)) return rc;
    if (int rc = check_workspace(op, workspace, workspace_bytes, convmi::gated_fwd_workspace(rows, C, F, dtype))) return rc;
    return gated_forward(op, x, w_gate, w_up, b_gate, b_up, h, saved, workspace, rows, C, F, act, dtype, stream);
}

int conv_gated_bwd_workspace_size(long long rows, int C, int F, int dtype, size_t* bytes)
{
    static const char* op = "conv_gated_bwd_workspace_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (int rc = check_gated(op, rows, C, F, CONV_ACT_NONE, dtype)) return rc;
    *bytes = convmi::gated_bwd_workspace(rows, C, F, dtype);
    return CONV_OK;
}

int conv_gated_bwd(const void* dh, const void* x, const void* w_gate, const void* w_up, const void* b_gate,
                   const void* b_up, const float* saved, void* dx, void* dw_gate, void* dw_up, void* db_gate, void* db_up,
                   void* workspace, size_t workspace_bytes, long long rows, int C, int F, int act, int dtype, void* stream)
{
    static const char* op = "conv_gated_bwd";
    if (int rc = check_gated(op, rows, C, F, act, dtype)) return rc;
    if (rows > 0 && (!dh || !x || !w_gate || !w_up))
        return fail(CONV_ERR_INVALID_ARG, "%s: dh, x, w_gate and w_up must not be NULL", op);
    if ((b_gate != nullptr) != (b_up != nullptr))
        return fail(CONV_ERR_INVALID_ARG, "%s: b_gate and b_up come together", op);
    if (int rc = check_aligned(op, {dh, x, w_gate, w_up, b_gate, b_up, dx, dw_gate, dw_up, db_gate, db_up},
                               dtype == CONV_F32 ? 4 : 2)) return rc;
    if (int rc = check_aligned(op, {saved}, 4)) return rc;
    if (int rc = check_workspace(op, workspace, workspace_bytes, convmi::gated_bwd_workspace(rows, C, F, dtype))) return rc;
    convmi::GatedArgs k{};
    k.dh = dh; k.x = x; k.wg = w_gate; k.wu = w_up; k.bg = b_gate; k.bu = b_up;
    k.saved = const_cast<float*>(saved);
    k.dx = dx; k.dwg = dw_gate; k.dwu = dw_up; k.dbg = db_gate; k.dbu = db_up;
    k.workspace = workspace;
    k.rows = rows; k.C = C; k.F = F; k.act = act;
    return launched(convmi::launch_gated_bwd(k, dtype, static_cast<hipStream_t>(stream)), op);
}

int conv_grad_workspace_size(int n, size_t* bytes)
{
    static const char* op = "conv_grad_workspace_size";
    if (!bytes) return fail(CONV_ERR_INVALID_ARG, "%s: bytes is NULL", op);
    if (n < 0) return fail(CONV_ERR_INVALID_ARG, "%s: n must be >= 0, got %d", op, n);
    *bytes = convmi::clip_workspace(n);
    return CONV_OK;
}

int conv_grad_norm(const void* const* grads, const size_t* counts, const int* dtypes, int n, float* norm,
                   void* workspace, size_t workspace_bytes, void* stream)
{
    static const char* op = "conv_grad_norm";
    if (!norm || off(norm, 4)) return fail(CONV_ERR_INVALID_ARG, "%s: norm must be a 4-byte aligned pointer", op);
    if (int rc = check_list(op, grads, nullptr, false, counts, dtypes, n, workspace, workspace_bytes)) return rc;
    return launched(convmi::launch_clip(grads, nullptr, counts, dtypes, n, 0.f, 0.f, norm, workspace,
                                        static_cast<hipStream_t>(stream)), op);
}

int conv_grad_clip(const void* const* grads, void* const* outs, const size_t* counts, const int* dtypes, int n,
                   float max_norm, float eps, float* norm, void* workspace, size_t workspace_bytes, void* stream)
{
    static const char* op = "conv_grad_clip";
    if (off(norm, 4)) return fail(CONV_ERR_INVALID_ARG, "%s: norm must be 4-byte aligned", op);
    if (!(max_norm >= 0.f) || !(eps >= 0.f) || !std::isfinite(eps))
        return fail(CONV_ERR_INVALID_ARG, "%s: max_norm and eps must be >= 0 and eps finite", op);
    if (int rc = check_list(op, grads, outs, true, counts, dtypes, n, workspace, workspace_bytes)) return rc;
    static void* const none[1] = {nullptr};
    return launched(convmi::launch_clip(grads, outs ? outs : none, counts, dtypes, n, max_norm, eps, norm, workspace,
                                        static_cast<hipStream_t>(stream)), op);
}

}  // extern "C"
