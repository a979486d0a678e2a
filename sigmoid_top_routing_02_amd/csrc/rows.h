// Rows of values in a block's registers: loads, stores and sums over a row, and the
// sums over the rows of a block's partial rows.  What the norms share.
#pragma once

#include "device_math.h"
#include "lanes.h"
#include "streaming.h"

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf v = {(__bf16)a, (__bf16)b};          // round to nearest even, NaN stays NaN
    return __builtin_bit_cast(uint32_t, v);
}

// A row of d values lies in the NV * 8 registers of each of its threads as 8
// consecutive values at ((v * tpr) + t) * 8, t of tpr threads.  VEC: d % 8 == 0, so
// that each such 8 lie on 16 bytes and in the row or past it; otherwise the vector
// accesses are to addresses of the values' own alignment, which this GPU takes, and
// the row's last up to 7 values are accessed one by one (32768 rows of bf16 values
// with residual: 999 wide 59 us against 84 with one value an access throughout, 4095
// wide 305 against 494, but 100 wide 22 against 16; the backward of 131072 rows, 999
// wide, 345 against 766).
__device__ __forceinline__ int col_of(int v, int t, int tpr) { return (v * tpr + t) * 8; }

template <bool VEC> struct Aligned {                     // four words
    typedef uint32_t bf16 __attribute__((ext_vector_type(4)));
    typedef float f32 __attribute__((ext_vector_type(4)));
};
template <> struct Aligned<false> {
    typedef uint32_t bf16 __attribute__((ext_vector_type(4), aligned(2)));
    typedef float f32 __attribute__((ext_vector_type(4), aligned(4)));
};

// 8 values of a row (zero past its end).  f32 is uniform over the launch.
template <bool VEC>
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t row_off, int v, int t, int tpr, int d,
                                      float (&x)[8]) {
    const int c = col_of(v, t, tpr);
    if (VEC ? c < d : c + 8 <= d) {
        if (f32) {
            const auto* q = reinterpret_cast<const typename Aligned<VEC>::f32*>(static_cast<const float*>(p) + row_off + c);
            const v4f a = q[0], b = q[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const v4u a = *reinterpret_cast<const typename Aligned<VEC>::bf16*>(static_cast<const uint16_t*>(p) + row_off + c);
            x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
            x[4] = bf16_lo(a.z); x[5] = bf16_hi(a.z); x[6] = bf16_lo(a.w); x[7] = bf16_hi(a.w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = VEC || c + j >= d ? 0.0f
                   : f32             ? static_cast<const float*>(p)[row_off + c + j]
                                     : bf16_to_f32(static_cast<const uint16_t*>(p)[row_off + c + j]);
    }
}

// (not through put(): a template's argument drops the vector types' lower alignment)
template <bool VEC, bool NT>
__device__ __forceinline__ void store8(void* p, bool f32, int64_t row_off, int v, int t, int tpr, int d,
                                       const float (&x)[8]) {
    const int c = col_of(v, t, tpr);
    if (VEC ? c < d : c + 8 <= d) {
        if (f32) {
            typedef typename Aligned<VEC>::f32 V;
            V* q = reinterpret_cast<V*>(static_cast<float*>(p) + row_off + c);
            const V a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
            if constexpr (NT) {
                __builtin_nontemporal_store(a, q);
                __builtin_nontemporal_store(b, q + 1);
            } else {
                q[0] = a;
                q[1] = b;
            }
        } else {
            typedef typename Aligned<VEC>::bf16 V;
            V* q = reinterpret_cast<V*>(static_cast<uint16_t*>(p) + row_off + c);
            const V a = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
            if constexpr (NT) __builtin_nontemporal_store(a, q);
            else *q = a;
        }
    } else if (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c + j >= d) continue;
            if (f32) static_cast<float*>(p)[row_off + c + j] = x[j];
            else static_cast<uint16_t*>(p)[row_off + c + j] = (uint16_t)pack_bf16(x[j], 0.0f);
        }
    }
}

// y rounded to bf16 and its 1x128 E4M3 tiles: 8 values at column c of a row of d,
// d % 128 == 0, so that 16 lanes are one tile, all in the row or none.
__device__ __forceinline__ void store_quant8(uint8_t* q, float* scale, int64_t row, int d, int c, int t, float (&y)[8]) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint32_t b = pack_bf16(y[j], y[j + 1]);
        y[j] = bf16_lo(b);
        y[j + 1] = bf16_hi(b);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float m = __builtin_fabsf(y[j]);
        amax = m > amax ? m : amax;
    }
    amax = max16(amax);
    float inv, sc;
    tile_scale(amax, inv, sc);
    if (c < d) {
        put<true>(reinterpret_cast<v2u*>(q + row * d + c),
                v2u{e4m3_encode4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                    e4m3_encode4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv)});
        if ((t & 15) == 0) scale[row * (d / 128) + c / 128] = sc;
    }
}

// Sum over the threads of one row: the wave by shuffles, the waves through LDS
// (two buffers in turn, so one barrier per row is enough).  Same order on every
// run.
template <bool WAVE_ROW>
__device__ __forceinline__ float row_sum(float s, float (*part)[16], int flip) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if constexpr (WAVE_ROW) return s;
    const int nw = (int)blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = s;
    // a barrier for LDS alone: loads and stores under way go on
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    s = part[flip][0];
    for (int i = 1; i < nw; ++i) s += part[flip][i];
    return s;
}

// Two such sums at once over a block's row, the waves' by wave_sum.
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*part)[16]) {
    a = wave_sum(a);
    b = wave_sum(b);
    if ((threadIdx.x & 63) == 0) {
        part[0][threadIdx.x >> 6] = a;
        part[1][threadIdx.x >> 6] = b;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int w = threadIdx.x & 15;                   // 16 lanes hold one wave's each
    const bool in = w < (int)blockDim.x >> 6;
    a = sum16(in ? part[0][w] : 0.0f);
    b = sum16(in ? part[1][w] : 0.0f);
}

// The sum in pairs, pairs of pairs and so on: a term goes through log2 N roundings.
template <int N>
__device__ __forceinline__ float pairwise(const float (&x)[N]) {
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = x[i];
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = s[2 * i] + s[2 * i + 1];
    return s[0];
}

// dw[c] = sum of the partial rows, pairwise: 16 threads take every 16th row of a
// column, eight loads at a time, then their sums are added (512 rows of 7168: 6 us,
// in which two blocks read every line, the 64 bytes of a row that one takes being half).
// Added one after the other they took the same time and left dw 1.2 to 2.1 times the
// error (32768 rows of 2048 FP32 values: 2.4e-7 of it, now 1.2e-7).
constexpr int MOST_PARTIAL_ROWS = 2048;                  // of backward_most
// The blocks of blockIdx.y = 1 do the same for db, whose partial rows follow dw's.
__global__ __launch_bounds__(256) void dw_reduce_kernel(const float* __restrict__ part, int rows, int d,
                                                        float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float sum[16][17];
    if (blockIdx.y) {
        part += (int64_t)rows * d;
        dw = db;
    }
    const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + cl;
    float s[MOST_PARTIAL_ROWS / 128];
#pragma unroll
    for (int k = 0; k < MOST_PARTIAL_ROWS / 128; ++k) {
        s[k] = 0.0f;
        if (k * 128 < rows && c < d) {
            const int r = k * 128 + rl;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = part[(int64_t)min(r + 16 * i, rows - 1) * d + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = r + 16 * i < rows ? x[i] : 0.0f;
            s[k] = pairwise(x);
        }
    }
    sum[rl][cl] = pairwise(s);
    __syncthreads();
    if (rl == 0 && c < d) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = sum[i][cl];
        dw[c] = pairwise(x);
    }
}

}  // namespace
}  // namespace moe
