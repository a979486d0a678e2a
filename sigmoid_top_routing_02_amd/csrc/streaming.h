// Stores of outputs that are written once and read by a later kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace moe {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <bool NT, typename T>
__device__ __forceinline__ void put(T* p, T v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Whether an output of so many bytes is stored non-temporally, so that it does not
// push the inputs out of the caches on its way: worth it where the output would
// not stay in the card's 256 MiB memory-side cache for its reader anyway.  Measured
// on rows of 7168 bf16 values, stored so / plainly: mxfp4_quant_1x32 with 30 MiB
// of output 25.4 / 23.3 us, 60 MiB 48 / 46, 120 MiB 92 / 100, 240 MiB 185 / 201;
// mxfp4_dequant_1x32 and a quantisation that reads its output, 14 MiB 9.0 / 9.9,
// 56 MiB 26.6 / 25.0, 448 MiB 200 / 226; the norm's backward and such a reader,
// 7 MiB 21.2 / 20.2, 56 MiB 73.7 / 71.3, alone with 896 MiB 746 / 769, and with
// rows of 512 values and 128 MiB 87 / 117.
inline bool streamed(int64_t bytes) { return bytes > ((int64_t)64 << 20); }

}  // namespace moe
