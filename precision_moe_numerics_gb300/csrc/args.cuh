// args.cuh -- what the C entry points ask of the addresses that they are given.
#pragma once
#include <cstdint>
#include <initializer_list>

namespace pmn {

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether p is one of the others' addresses (NULL: a tensor that is not there).
inline bool among(const void *p, std::initializer_list<const void *> others)
{
    for (const void *q : others)
        if (p && p == q) return true;
    return false;
}

}  // namespace pmn
