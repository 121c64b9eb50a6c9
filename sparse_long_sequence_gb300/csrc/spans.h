// Argument checks that the operators' entry points share: a call's tensors as spans of bytes.
#pragma once

#include <cstdint>
#include <string>

#include "internal.h"

namespace dfs {

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// A tensor of a call: where it is and how many bytes.
struct Span {
    const void* p;
    size_t bytes;
};

inline int check_span(const Span& s, const char* what, size_t align = 16) {
    if (s.bytes && !s.p) return fail(DIFFUSER_ERR_INVALID_ARG, std::string(what) + " is NULL");
    if (reinterpret_cast<uintptr_t>(s.p) % align)
        return fail(DIFFUSER_ERR_INVALID_ARG, std::string(what) + " is not " + std::to_string(align) + "-byte aligned");
    return DIFFUSER_OK;
}
inline bool meets(const Span& a, const Span& b) {
    return a.p && b.p && a.bytes && b.bytes && overlaps(a.p, a.bytes, b.p, b.bytes);
}

// Outputs (null ones are left out) may overlap no input and no other output, but
// output `in_place[o]` may be exactly input number in_place[o] (-1: none).
inline int check_overlaps(const Span* in, int nin, const Span* out, int nout, const int* in_place = nullptr) {
    for (int o = 0; o < nout; ++o) {
        for (int x = 0; x < nin; ++x) {
            if (in_place && in_place[o] == x && in[x].p == out[o].p) continue;
            if (meets(out[o], in[x])) return fail(DIFFUSER_ERR_INVALID_ARG, "an output overlaps an input");
        }
        for (int x = o + 1; x < nout; ++x)
            if (meets(out[o], out[x])) return fail(DIFFUSER_ERR_INVALID_ARG, "the outputs overlap");
    }
    return DIFFUSER_OK;
}

}  // namespace dfs
