// fl_check.hpp -- host side: the error message of a unit's entry points and
// the checks of their arguments.  Every unit that includes it has a message of
// its own, thread-local.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "fused_linear.h"

namespace {

thread_local char g_err[512];

fl_status fail(fl_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}

void clear_error() { g_err[0] = '\0'; }

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr size_t kTwoGiB = 0x80000000ull;

size_t elem_size(int dtype) { return dtype == FL_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (!a || !b || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

// An operand of a call: name, bytes it spans, alignment; `out` is written.
struct Operand {
    const char *name;
    const void *p;
    size_t bytes, align;
    bool out, optional;
    const void *same;  // an input this output may equal exactly
};

template <int N>
fl_status check_operands(const Operand (&ops)[N]) {
    for (const Operand &o : ops) {
        if (!o.p && o.bytes && !o.optional) return fail(FL_ERR_INVALID_ARG, "%s is NULL", o.name);
        if (o.p && !aligned(o.p, o.align))
            return fail(FL_ERR_INVALID_ARG, "%s (%p) is not aligned to %zu bytes", o.name, o.p, o.align);
    }
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            const Operand &o = ops[i], &q = ops[j];
            if (i == j || !o.out || (q.out && j < i)) continue;
            if (!q.out && o.same && o.p == q.p && o.same == q.p) continue;
            if (overlaps(o.p, o.bytes, q.p, q.bytes))
                return fail(FL_ERR_INVALID_ARG, "%s overlaps %s", o.name, q.name);
        }
    return FL_OK;
}

template <int N>
fl_status check_sizes(const int64_t (&v)[N]) {
    for (int64_t x : v)
        if (x < 0) return fail(FL_ERR_INVALID_ARG, "negative size %lld", (long long)x);
    for (int64_t x : v)
        if (x > kMaxDim) return fail(FL_ERR_UNSUPPORTED, "sizes above 2^31-1 are not supported");
    return FL_OK;
}

fl_status check_dtype(int d) {
    return d == FL_F32 || d == FL_F16 || d == FL_BF16 ? FL_OK : fail(FL_ERR_INVALID_ARG, "unknown dtype %d", d);
}

fl_status check_launch(const char *what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(FL_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
    return FL_OK;
}

}  // namespace
