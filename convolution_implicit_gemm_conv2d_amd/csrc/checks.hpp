// Checks of arguments that the C entry points share.  They run on the host
// before anything is launched.
#pragma once

#include "act.hpp"
#include "convmi.h"
#include "kernels.hpp"

#include <algorithm>
#include <cstdint>

namespace convmi {
namespace checks {

constexpr int kMaxWidth = 1 << 20;  // channels of a row

inline bool off(const void* p, size_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

inline int check_dtype(const char* op, int dtype)
{
    if (dtype != CONV_F32 && dtype != CONV_BF16)
        return fail(CONV_ERR_INVALID_ARG, "%s: dtype must be CONV_F32 or CONV_BF16, got %d", op, dtype);
    return CONV_OK;
}

inline int check_sizes(const char* op, long long rows, long long C, const char* name)
{
    if (rows < 0 || C < 1)
        return fail(CONV_ERR_INVALID_ARG, "%s: rows must be >= 0 and %s >= 1 (got %lld, %lld)", op, name, rows, C);
    if (rows > INT32_MAX || C > kMaxWidth)
        return fail(CONV_ERR_OVERFLOW, "%s: rows must be below 2^31 and %s at most 2^20 (got %lld, %lld)", op, name, rows, C);
    return CONV_OK;
}

inline int check_aligned(const char* op, std::initializer_list<const void*> tensors, size_t align)
{
    for (const void* p : tensors)
        if (off(p, align))
            return fail(CONV_ERR_INVALID_ARG, "%s: a tensor is not aligned to its %zu-byte elements", op, align);
    return CONV_OK;
}

inline int check_workspace(const char* op, const void* workspace, size_t bytes, size_t need)
{
    if (bytes < need || (need > 0 && (!workspace || off(workspace, 16))))
        return fail(CONV_ERR_INVALID_ARG, "%s: needs a 16-byte aligned workspace of %zu bytes (got %zu)", op, need, bytes);
    return CONV_OK;
}

inline int launched(hipError_t e, const char* op)
{
    return e == hipSuccess ? CONV_OK : fail(CONV_ERR_HIP, "%s: launch failed: %s", op, hipGetErrorString(e));
}

inline int check_act(const char* op, int act)
{
    if (act < 0 || act >= convmi::kActs) return fail(CONV_ERR_INVALID_ARG, "%s: %d is not a conv_act_t", op, act);
    return CONV_OK;
}

// The memory of one tensor of a list.
struct Span {
    uintptr_t at, end;
    bool written;
};

// No written span meets another one.  Sorts them.
inline bool spans_apart(Span* s, int m)
{
    std::sort(s, s + m, [](const Span& a, const Span& b) { return a.at < b.at; });
    uintptr_t any = 0, written = 0;  // how far the spans up to here reach
    for (int i = 0; i < m; ++i) {
        if (s[i].at < (s[i].written ? any : written)) return false;
        any = std::max(any, s[i].end);
        if (s[i].written) written = std::max(written, s[i].end);
    }
    return true;
}

}  // namespace checks
}  // namespace convmi
