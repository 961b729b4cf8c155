// operands.h -- checks of the arrays that an entry point takes.
#pragma once

#include <cstddef>
#include <cstdint>

#include "aggraph.h"
#include "internal.h"

namespace ag {
namespace {

constexpr int kCurrent = -1;

// Inputs that a row-wise kernel reads an element of in the thread that writes
// the output's (matrices), inputs that several rows read (parameters), outputs,
// outputs of a launch that follows on all reads, and scratch.  Maybe: may be null.
enum Role { kIn, kMaybeIn, kParam, kMaybeParam, kOut, kMaybeOut, kMaybeLast, kMaybeScratch };

struct Operand {
    const void *p;
    const char *name;
    size_t bytes;
    int align;
    Role role;
    bool output() const { return role >= kOut; }
    bool needed() const { return role == kIn || role == kParam || role == kOut; }
    // whether this output may lie exactly where the input x does
    bool in_place_of(const Operand &x) const {
        if (x.output() || x.p != p || x.bytes != bytes || role == kMaybeScratch) return false;
        return role == kMaybeLast || x.role == kIn || x.role == kMaybeIn;
    }
};

// Every array given where it has to be, aligned to its elements, of `device`
// (kCurrent: the calling thread's, for calls without a graph).
// An output shares no memory with an output, and with an input none, or
// (in_place) all of a matrix: the row-wise kernels read an element before they
// write it, in the thread that writes it.
template <int K>
int check_operands(const Operand (&a)[K], int device, bool in_place, const char *fn) {
    for (const Operand &x : a) {
        if (!x.p && x.needed()) return fail(AG_ERR_INVALID_ARG, "%s: null %s", fn, x.name);
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
            if (in_place && a[i].in_place_of(a[j])) continue;
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
