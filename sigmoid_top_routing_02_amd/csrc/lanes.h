// Reductions over the lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Sums and maxima over lanes without LDS: within 16 lanes by DPP (neighbours, pairs,
// halves, all 16 mirrored), then over the wave's four sixteens by lane swaps.  Every
// lane gets the same bits.  (A row of LDS shuffles is six times their latency.)
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float s) {
    s += dpp<0xB1>(s);                                // quad_perm 1 0 3 2
    s += dpp<0x4E>(s);                                // quad_perm 2 3 0 1
    s += dpp<0x141>(s);                               // row_half_mirror
    return s + dpp<0x140>(s);                         // row_mirror
}
__device__ __forceinline__ float wave_sum(float s) {
    s = sum16(s);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    s = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// over each L = 16, 32 or 64 lanes
template <int L>
__device__ __forceinline__ float lanes_sum(float s) {
    if constexpr (L == 64) return wave_sum(s);
    s = sum16(s);
    if constexpr (L == 16) return s;
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float max16(float m) {     // a NaN counts as less than anything
    float o = dpp<0xB1>(m);
    m = o > m ? o : m;
    o = dpp<0x4E>(m);
    m = o > m ? o : m;
    o = dpp<0x141>(m);
    m = o > m ? o : m;
    o = dpp<0x140>(m);
    return o > m ? o : m;
}

// the least over each L = 16 or 64 lanes
template <int L>
__device__ __forceinline__ int lanes_min(int m) {
    auto with = [&](int o) { m = o < m ? o : m; };
    with(__builtin_amdgcn_update_dpp(m, m, 0xB1, 0xf, 0xf, false));       // the lanes of sum16
    with(__builtin_amdgcn_update_dpp(m, m, 0x4E, 0xf, 0xf, false));
    with(__builtin_amdgcn_update_dpp(m, m, 0x141, 0xf, 0xf, false));
    with(__builtin_amdgcn_update_dpp(m, m, 0x140, 0xf, 0xf, false));
    if constexpr (L == 64) {
        const auto a = __builtin_amdgcn_permlane16_swap((unsigned)m, (unsigned)m, false, false);
        m = (int)a[0] < (int)a[1] ? (int)a[0] : (int)a[1];
        const auto b = __builtin_amdgcn_permlane32_swap((unsigned)m, (unsigned)m, false, false);
        m = (int)b[0] < (int)b[1] ? (int)b[0] : (int)b[1];
    }
    return m;
}

// the largest of lanes l, l ^ 16, l ^ 32 and l ^ 48 (of no NaN)
__device__ __forceinline__ float max_of_rows(float m) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = __uint_as_float(a[0]) > __uint_as_float(a[1]) ? __uint_as_float(a[0]) : __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return __uint_as_float(b[0]) > __uint_as_float(b[1]) ? __uint_as_float(b[0]) : __uint_as_float(b[1]);
}

}  // namespace moe
