// host.hpp -- host-side pieces shared by the library's translation units:
// the per-device compute-unit count, launches, and argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>
#include <stdint.h>

#include "gemm355.h"

namespace gemm355 {
namespace host {

constexpr int kMaxDevices = 64;

inline std::mutex g_cu_lock;
inline int g_cu_count[kMaxDevices];   // 0 = not queried yet

// Compute units of the current device, queried once per device.
inline int compute_units(int *cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return GEMM355_ERR_NO_DEVICE;
    std::lock_guard<std::mutex> guard(g_cu_lock);
    if (g_cu_count[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
            return GEMM355_ERR_NO_DEVICE;
        g_cu_count[dev] = n;
    }
    *cus = g_cu_count[dev];
    return GEMM355_OK;
}

// One kernel launch on `stream`. The launch's own return code is the status:
// the thread's pending HIP error is neither read nor cleared, so an error the
// caller has not collected yet stays theirs.
template <class Kernel, class Args>
int launch_kernel(Kernel kernel, unsigned blocks, unsigned threads, Args &args, hipStream_t stream)
{
    void *argv[] = {&args};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(blocks), dim3(threads), argv,
                                         0, stream);
    return e == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlaps(const void *p, size_t pn, const void *q, size_t qn)
{
    if (!p || !q || pn == 0 || qn == 0)
        return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qn && b < a + pn;
}

// Byte extent of `rows` rows (rounded up to whole 256-row tiles) of `row_bytes`
// each must stay below 2^31: the kernels address operands with 32-bit offsets.
inline bool extent_ok(int64_t rows, int64_t row_bytes)
{
    const int64_t padded = (rows + 255) / 256 * 256;
    return padded * row_bytes < (int64_t(1) << 31);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

} // namespace host
} // namespace gemm355
