// Argument checks shared by the host files of the C ABI (ck_api.cpp,
// ck_rows_api.cpp and ck_fp8_api.cpp).  Plain host C++ without HIP calls, allocations or exceptions:
// a failed check writes the thread's error message and returns a status.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "../../include/ck.h"

namespace ck {
namespace api {

inline thread_local char g_last_error[512] = "";

inline int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return status;
}

inline int ok()
{
    g_last_error[0] = '\0';
    return CK_OK;
}

inline int hip_status(int e, const char *what)
{
    if (e != 0)
        return fail(CK_ERR_HIP, "%s: HIP launch failed (hipError_t %d)", what, e);
    return ok();
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte range [lo, hi) spanned by `rows` rows of `cols` elements of `esize`
// bytes with row stride `ld` elements.
struct Range {
    uintptr_t lo = 0, hi = 0;
};
inline Range span(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esize)
{
    Range r;
    if (!p || rows <= 0 || cols <= 0)
        return r;
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + (uintptr_t)(((rows - 1) * ld + cols) * esize);
    return r;
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

constexpr int64_t kMaxK = 32768;
// A launch covers at most 2^32 - 1 work-items per grid dimension.  Rotate-quant
// and the weight producer launch one workgroup of up to 1024 threads per row,
// so the rows stay below 2^22: (2^22 - 1) * 1024 = 2^32 - 1024 work-items.
constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;

inline int check_k(const char *fn, int64_t K)
{
    if (K <= 0)
        return fail(CK_ERR_INVALID_ARG, "%s: K must be positive (got %lld)", fn, (long long)K);
    if (K % 64 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: K must be a multiple of 64 (got %lld)", fn, (long long)K);
    if (K > kMaxK)
        return fail(CK_ERR_UNSUPPORTED, "%s: K must be at most %lld (got %lld)", fn, (long long)kMaxK,
                    (long long)K);
    return CK_OK;
}

inline int check_m(const char *fn, int64_t M)
{
    if (M < 0)
        return fail(CK_ERR_INVALID_ARG, "%s: M must be >= 0 (got %lld)", fn, (long long)M);
    if (M > kMaxRows)
        return fail(CK_ERR_UNSUPPORTED, "%s: M above %lld", fn, (long long)kMaxRows);
    return CK_OK;
}

inline int check_x(const char *fn, const uint16_t *x, int64_t K, int64_t ldx)
{
    if (!x)
        return fail(CK_ERR_INVALID_ARG, "%s: x is NULL", fn);
    if (ldx < K || ldx % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: ldx (%lld) must be >= K and a multiple of 8", fn,
                    (long long)ldx);
    if (!aligned(x, 16))
        return fail(CK_ERR_INVALID_ARG, "%s: x must be 16-byte aligned", fn);
    return CK_OK;
}

// Outputs are written with 16-byte stores: 16-byte aligned rows.
inline int check_out(const char *fn, const void *out, int64_t N, int64_t ldo, size_t esize)
{
    if (!out)
        return fail(CK_ERR_INVALID_ARG, "%s: output is NULL", fn);
    const int64_t per16 = 16 / (int64_t)esize;
    if (ldo < N || ldo % per16 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: output stride (%lld) must be >= N and a multiple of %lld",
                    fn, (long long)ldo, (long long)per16);
    if (!aligned(out, 16))
        return fail(CK_ERR_INVALID_ARG, "%s: output must be 16-byte aligned", fn);
    return CK_OK;
}

#define CK_TRY(expr)            \
    do {                        \
        int _st = (expr);       \
        if (_st != CK_OK)       \
            return _st;         \
    } while (0)

constexpr size_t kWsAlign = 256;
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace api
}  // namespace ck
