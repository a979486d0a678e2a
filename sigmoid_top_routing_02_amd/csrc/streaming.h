// Stores of outputs that are written once and read by a later kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <bool NT, typename T>
__device__ __forceinline__ void put(T* p, T v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Whether an output of so many bytes is stored past L2 (non-temporal): where it is
// larger than the 32 MiB of L2 on the card, most of it would be written back
// before the next kernel could read it there.
inline bool stored_past_l2(int64_t bytes) { return bytes > ((int64_t)32 << 20); }

}  // namespace moe
