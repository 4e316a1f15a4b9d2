// abi_checks.cuh -- what the C entry points of the token policy's layers and
// losses check before they launch (host side only).
#pragma once

#include <initializer_list>

#include "residency.cuh"
#include "sequence.cuh"

namespace rlscan {
namespace seq {

inline cudaStream_t cs(rlscan_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool equals_any(const void *out, std::initializer_list<const void *> others)
{
    for (const void *o : others)
        if (o != nullptr && o == out) return true;
    return false;
}

// the residency of all of them together: the one that allows least
inline Residency residency_of(std::initializer_list<const void *> ptrs)
{
    Residency all = Residency::Device;
    for (const void *p : ptrs) {
        const Residency one = p != nullptr ? residency(p) : Residency::Device;
        if (one == Residency::Unreachable) return one;
        if (one == Residency::Host) all = one;
    }
    return all;
}
inline bool reachable(std::initializer_list<const void *> ptrs) { return residency_of(ptrs) != Residency::Unreachable; }
// Copies into shared memory are for device memory alone.
inline bool on_device(std::initializer_list<const void *> ptrs) { return residency_of(ptrs) == Residency::Device; }

inline bool workspace_ok(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws != nullptr && have >= need && (reinterpret_cast<uintptr_t>(ws) & 15u) == 0 &&
                         residency(ws) == Residency::Device);
}

inline bool is_io_type(int64_t t) { return t == RLSCAN_F32 || t == RLSCAN_BF16; }

// sizes whose products stay far inside 63 bits, and grids inside 31
inline bool sizes_ok(std::initializer_list<int64_t> sizes)
{
    double all = 1;
    for (int64_t v : sizes) {
        if (v < 0) return false;
        all *= v > 0 ? static_cast<double>(v) : 1.0;
    }
    return all < 1e15;
}

}  // namespace seq
}  // namespace rlscan

#define RLSCAN_TRY(expr)                           \
    do {                                           \
        const rlscan_status st_ = (expr);          \
        if (st_ != RLSCAN_OK) return st_;          \
    } while (0)

#define RLSCAN_API __attribute__((visibility("default")))
