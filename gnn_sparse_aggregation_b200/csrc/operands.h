// operands.h -- checks of the arrays that an entry point takes.
#pragma once

#include <cstddef>
#include <cstdint>

#include "aggraph.h"
#include "internal.h"

namespace ag {
namespace {

constexpr int kCurrent = -1;

enum Role { kIn, kMaybeIn, kOut, kMaybeOut };  // input, input that may be null, output, output that may be null

struct Operand {
    const void *p;
    const char *name;
    size_t bytes;
    int align;
    Role role;
    bool output() const { return role == kOut || role == kMaybeOut; }
};

// Every array given where it has to be, aligned to its elements, of `device`
// (kCurrent: the calling thread's, for calls without a graph).
// An output shares no memory with an output, and with an input none, or
// (in_place) all of it: the row-wise kernels read an element before they write
// it, in the thread that writes it.
template <int K>
int check_operands(const Operand (&a)[K], int device, bool in_place, const char *fn) {
    for (const Operand &x : a) {
        if (!x.p && (x.role == kIn || x.role == kOut)) return fail(AG_ERR_INVALID_ARG, "%s: null %s", fn, x.name);
        if (reinterpret_cast<uintptr_t>(x.p) % uintptr_t(x.align) != 0)
            return fail(AG_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, x.name);
    }
    for (int i = 0; i < K; ++i) {
        if (!a[i].p || !a[i].output()) continue;
        const uintptr_t b = reinterpret_cast<uintptr_t>(a[i].p);
        for (int j = 0; j < K; ++j) {
            if (j == i || !a[j].p) continue;
            const uintptr_t c = reinterpret_cast<uintptr_t>(a[j].p);
            if (b >= c + a[j].bytes || c >= b + a[i].bytes) continue;
            if (in_place && !a[j].output() && b == c && a[i].bytes == a[j].bytes) continue;
            return fail(AG_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, a[i].name, a[j].name);
        }
    }
    if (device == kCurrent) {
        cudaError_t err = cudaGetDevice(&device);
        if (err != cudaSuccess) return cuda_fail(err, fn);
    }
    for (const Operand &x : a)
        if (x.p)
            if (int rc = check_device_ptr(x.p, device, x.name)) return rc;
    return AG_OK;
}

}  // namespace
}  // namespace ag
