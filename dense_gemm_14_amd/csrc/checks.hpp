// checks.hpp -- checks of a call's arrays, shared by the host files of the calls
// that take several outputs and a workspace.
#pragma once

#include "host.hpp"

namespace gemm355 {
namespace host {

// An array of a call: its address and size.
struct Array {
    const void *p;
    size_t bytes;
};

// Whether any output overlaps an input, the workspace or another output.
inline bool any_overlap(const Array *out, int outs, const Array *in, int ins)
{
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return true;
        for (int j = i + 1; j < outs; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return true;
    }
    return false;
}

inline bool all_aligned(const Array *a, int n)
{
    for (int i = 0; i < n; ++i)
        if (!aligned(a[i].p, 16))
            return false;
    return true;
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

} // namespace host
} // namespace gemm355
