// C ABI of the optimizer step: argument checks and launches.  Every check runs
// on the host before anything is launched.
#include "checks.hpp"

#include <cmath>
#include <memory>
#include <new>

using namespace convmi::checks;
using convmi::fail;

namespace {

size_t size_of(int dtype) { return dtype == CONV_F32 ? 4 : 2; }

size_t scale_bytes(int, size_t c) { return (c + convmi::kAdamBlock - 1) / convmi::kAdamBlock * 4; }

// Spans of a call's lists, to be told apart: list after list, since each mostly
// ascends already and is sorted sooner so (468 tensors with 8-bit states: 23 us,
// and 91 us tensor after tensor).
struct Spans {
    static constexpr int kHere = 512;
    Span here[kHere];
    std::unique_ptr<Span[]> more;
    Span* s = here;
    int m = 0;

    bool room(int64_t n)
    {
        if (n <= kHere) return true;
        more.reset(new (std::nothrow) Span[static_cast<size_t>(n)]);
        s = more.get();
        return s != nullptr;
    }
    void add(const void* p, size_t bytes, bool written)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        if (bytes) s[m++] = Span{at, at + bytes, written};
    }
    template <typename P, typename F>
    void list(const P* p, const size_t* counts, int n, F bytes, bool written)
    {
        for (int i = 0; i < n; ++i)
            if (counts[i]) add(p[i], bytes(i, counts[i]), written);
    }
};

bool number(double v, double least) { return v >= least && std::isfinite(v) && std::isfinite(static_cast<float>(v)); }

}  // namespace

extern "C" {

int conv_adamw(void* const* params, const void* const* grads, void* const* m, void* const* v, float* const* m_scales, float* const* v_scales,
               void* const* copies, const size_t* counts, const int* param_dtypes, const int* grad_dtypes, const int* copy_dtypes, int n, int bits,
               double lr, double beta1, double beta2, double eps, double weight_decay, long long step, const float* lr_dev, const long long* step_dev,
               const float* norm, double max_norm, double norm_eps, void* stream)
{
    static const char* op = "conv_adamw";
    if (n < 0) return fail(CONV_ERR_INVALID_ARG, "%s: n must be >= 0, got %d", op, n);
    if (bits != 8 && bits != 32) return fail(CONV_ERR_INVALID_ARG, "%s: bits must be 8 or 32, got %d", op, bits);
    if (n > 0 && (!params || !grads || !m || !v || !counts || !param_dtypes || !grad_dtypes || (bits == 8 && (!m_scales || !v_scales)) || (copies && !copy_dtypes)))
        return fail(CONV_ERR_INVALID_ARG, "%s: an array is NULL", op);
    if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1) || static_cast<float>(beta1) >= 1.f || static_cast<float>(beta2) >= 1.f)
        return fail(CONV_ERR_INVALID_ARG, "%s: beta1 and beta2 must be in [0, 1)", op);
    if (!number(eps, 0x1p-126) || !number(weight_decay, 0) || !number(max_norm, 0) || !number(norm_eps, 0) || !std::isfinite(lr) ||
        !std::isfinite(static_cast<float>(lr)))
        return fail(CONV_ERR_INVALID_ARG, "%s: lr, eps (from 2^-126 on), weight_decay, max_norm and norm_eps must be finite and the last four not negative", op);
    if (!step_dev && step < 1) return fail(CONV_ERR_INVALID_ARG, "%s: step counts from 1, got %lld", op, step);
    if (off(lr_dev, 4) || off(step_dev, 8) || off(norm, 4)) return fail(CONV_ERR_INVALID_ARG, "%s: lr_dev, step_dev or norm is misaligned", op);
    Spans s;
    if (!s.room(7 * static_cast<int64_t>(n) + 3)) return fail(CONV_ERR_HIP, "%s: no host memory to check %d tensors", op, n);
    for (int i = 0; i < n; ++i) {
        if (int rc = check_dtype(op, param_dtypes[i])) return rc;
        if (int rc = check_dtype(op, grad_dtypes[i])) return rc;
        const bool copied = copies && copies[i];
        if (copied)
            if (int rc = check_dtype(op, copy_dtypes[i])) return rc;
        const size_t c = counts[i];
        if (c == 0) continue;
        if (c >> 38) return fail(CONV_ERR_OVERFLOW, "%s: tensor %d has 2^38 elements or more", op, i);
        if (!params[i] || !grads[i] || !m[i] || !v[i] || (bits == 8 && (!m_scales[i] || !v_scales[i])))
            return fail(CONV_ERR_INVALID_ARG, "%s: a pointer of tensor %d is NULL", op, i);
        const size_t ps = size_of(param_dtypes[i]), gs = size_of(grad_dtypes[i]), cs = copied ? size_of(copy_dtypes[i]) : 1;
        if (off(params[i], ps) || off(grads[i], gs) || (copied && off(copies[i], cs)) || (bits == 32 && (off(m[i], 4) || off(v[i], 4))) ||
            (bits == 8 && (off(m_scales[i], 4) || off(v_scales[i], 4))))
            return fail(CONV_ERR_INVALID_ARG, "%s: a pointer of tensor %d is not aligned to its elements", op, i);
    }
    s.list(params, counts, n, [&](int i, size_t c) { return c * size_of(param_dtypes[i]); }, true);
    s.list(grads, counts, n, [&](int i, size_t c) { return c * size_of(grad_dtypes[i]); }, false);
    s.list(m, counts, n, [&](int, size_t c) { return c * (bits / 8); }, true);
    s.list(v, counts, n, [&](int, size_t c) { return c * (bits / 8); }, true);
    if (copies) s.list(copies, counts, n, [&](int i, size_t c) { return copies[i] ? c * size_of(copy_dtypes[i]) : 0; }, true);
    if (bits == 8) {
        s.list(m_scales, counts, n, scale_bytes, true);
        s.list(v_scales, counts, n, scale_bytes, true);
    }
    if (lr_dev) s.add(lr_dev, 4, false);
    if (step_dev) s.add(step_dev, 8, false);
    if (norm) s.add(norm, 4, false);
    if (!spans_apart(s.s, s.m)) return fail(CONV_ERR_INVALID_ARG, "%s: what is written overlaps another tensor of the call", op);
    const convmi::AdamList l{params, m, v, copies, grads, m_scales, v_scales, counts, param_dtypes, grad_dtypes, copy_dtypes, n, bits};
    const convmi::AdamRates r{lr, beta1, beta2, eps, weight_decay, max_norm, norm_eps, step_dev ? 1 : step, lr_dev, norm, step_dev};
    return launched(convmi::launch_adamw(l, r, static_cast<hipStream_t>(stream)), op);
}

int conv_adamw_moments(const void* const* m, const void* const* v, const float* const* m_scales, const float* const* v_scales, float* const* m_out,
                       float* const* v_out, const size_t* counts, int n, void* stream)
{
    static const char* op = "conv_adamw_moments";
    if (n < 0) return fail(CONV_ERR_INVALID_ARG, "%s: n must be >= 0, got %d", op, n);
    if (n > 0 && (!m || !v || !m_scales || !v_scales || !m_out || !v_out || !counts)) return fail(CONV_ERR_INVALID_ARG, "%s: an array is NULL", op);
    Spans s;
    if (!s.room(6 * static_cast<int64_t>(n))) return fail(CONV_ERR_HIP, "%s: no host memory to check %d tensors", op, n);
    for (int i = 0; i < n; ++i) {
        const size_t c = counts[i];
        if (c == 0) continue;
        if (c >> 38) return fail(CONV_ERR_OVERFLOW, "%s: tensor %d has 2^38 elements or more", op, i);
        if (!m[i] || !v[i] || !m_scales[i] || !v_scales[i] || !m_out[i] || !v_out[i] || off(m_scales[i], 4) || off(v_scales[i], 4) || off(m_out[i], 4) ||
            off(v_out[i], 4))
            return fail(CONV_ERR_INVALID_ARG, "%s: a pointer of tensor %d is NULL or misaligned", op, i);
    }
    s.list(m, counts, n, [](int, size_t c) { return c; }, false);
    s.list(v, counts, n, [](int, size_t c) { return c; }, false);
    s.list(m_scales, counts, n, scale_bytes, false);
    s.list(v_scales, counts, n, scale_bytes, false);
    s.list(m_out, counts, n, [](int, size_t c) { return c * 4; }, true);
    s.list(v_out, counts, n, [](int, size_t c) { return c * 4; }, true);
    if (!spans_apart(s.s, s.m)) return fail(CONV_ERR_INVALID_ARG, "%s: what is written overlaps another tensor of the call", op);
    const convmi::AdamList l{nullptr, const_cast<void* const*>(m), const_cast<void* const*>(v), nullptr, nullptr, const_cast<float* const*>(m_scales),
                             const_cast<float* const*>(v_scales), counts, nullptr, nullptr, nullptr, n, 8};
    return launched(convmi::launch_adamw_moments(l, m_out, v_out, static_cast<hipStream_t>(stream)), op);
}

}  // extern "C"
