// MXFP4 (OCP microscaling: E2M1 codes, one E8M0 scale byte per 32 consecutive
// values) quantiser and dequantiser, and the 1x128 E4M3 dequantiser.
//
// Scale of a block: 2^e with e = floor(log2 amax) - 2, so that amax lands in
// [4, 8) and only values above 6 saturate; the byte is e + 127, clamped at 0
// (amax below 2^-124, zero included).  amax is found on the bit patterns, whose
// order is the magnitudes' order; a block that holds a NaN or an infinity
// (exponent field 255) gets the NaN scale 0xFF and zero codes, so that it stays
// visible: E2M1 has no code for either.  Codes are x / 2^e rounded to nearest,
// ties to even, by gfx950's conversion, which saturates at 6 and keeps signs.
//
// All three stream HBM: 8 values a lane, four lanes one block (the block's
// maximum is two lane exchanges), U steps of the whole grid in flight per lane.
#include "device_math.h"
#include "kernels.h"

namespace moe {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
constexpr int U = 4;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The float 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

template <bool IN_F32>
__global__ __launch_bounds__(256) void mxfp4_quant_kernel(const void* __restrict__ x, int64_t lanes,
                                                          uint32_t* __restrict__ q, uint8_t* __restrict__ scale) {
    // `lanes` is a multiple of 4 and so is every stride: the lanes of a block
    // are live together
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 + threadIdx.x; g0 - threadIdx.x < lanes; g0 += stride * U) {
        uint4 raw[U][IN_F32 ? 2 : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            const uint4* p = static_cast<const uint4*>(x) + (g < lanes ? g : 0) * (IN_F32 ? 2 : 1);
            raw[u][0] = p[0];
            if constexpr (IN_F32) raw[u][1] = p[1];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            uint32_t m;                                  // exponent field of the largest magnitude
            if constexpr (IN_F32) {
                const uint4 a = raw[u][0], b = raw[u][1];
                m = umax(umax(umax(a.x << 1, a.y << 1), umax(a.z << 1, a.w << 1)),
                         umax(umax(b.x << 1, b.y << 1), umax(b.z << 1, b.w << 1)));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64)) >> 24;
            } else {
                const uint4 a = raw[u][0];
                m = umax(umax(umax(a.x << 17, a.y << 17), umax(a.z << 17, a.w << 17)),
                         umax(umax(a.x & 0x7FFF0000u, a.y & 0x7FFF0000u), umax(a.z & 0x7FFF0000u, a.w & 0x7FFF0000u)) << 1);
                m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64)) >> 24;
            }
            const uint32_t byte = m == 255u ? 255u : m > 2u ? m - 2u : 0u;
            const float s = e8m0(byte == 255u ? 127u : byte);
            uint32_t w = 0;
            if constexpr (IN_F32) {
                const uint4 a = raw[u][0], b = raw[u][1];
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a.x), __uint_as_float(a.y), s, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a.z), __uint_as_float(a.w), s, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b.x), __uint_as_float(b.y), s, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b.z), __uint_as_float(b.w), s, 3);
            } else {
                const uint4 a = raw[u][0];
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, a.x), s, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, a.y), s, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, a.z), s, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, a.w), s, 3);
            }
            if (g < lanes) {
                q[g] = byte == 255u ? 0u : w;
                if ((g & 3) == 0) scale[g >> 2] = (uint8_t)byte;
            }
        }
    }
}

template <bool OUT_F32>
__device__ __forceinline__ void store_values(void* out, int64_t g, const float (&v)[8]) {
    if constexpr (OUT_F32) {
        float4* o = static_cast<float4*>(out) + g * 2;
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const v2bf b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, b);
        }
        static_cast<uint4*>(out)[g] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Exact: an E2M1 value times a power of two is a bf16 and a binary32 value
// (subnormals included), but for 4 and 6 times the scale 2^127, which no
// quantiser output has and which overflow to infinity.
template <bool OUT_F32>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint32_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scale, int64_t lanes,
                                                            void* __restrict__ out) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 + threadIdx.x; g0 < lanes; g0 += stride * U) {
        uint32_t w[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            w[u] = q[g < lanes ? g : 0];
            s[u] = scale[g < lanes ? g >> 2 : 0];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            if (g >= lanes) continue;
            const float sc = s[u] == 255u ? __builtin_nanf("") : e8m0(s[u]);
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0);
            const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
            const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2);
            const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
            const float v[8] = {a.x * sc, a.y * sc, b.x * sc, b.y * sc, c.x * sc, c.y * sc, d.x * sc, d.y * sc};
            store_values<OUT_F32>(out, g, v);
        }
    }
}

// E4M3(q) * scale in binary32, rounded once where the output is bf16.
template <bool OUT_F32>
__global__ __launch_bounds__(256) void fp8_dequant_1x128_kernel(const uint2* __restrict__ q,
                                                                const float* __restrict__ scale, int64_t lanes,
                                                                void* __restrict__ out) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 + threadIdx.x; g0 < lanes; g0 += stride * U) {
        uint2 w[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            w[u] = q[g < lanes ? g : 0];
            s[u] = scale[g < lanes ? g >> 4 : 0];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            if (g >= lanes) continue;
            const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u].x, false);
            const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u].x, true);
            const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u].y, false);
            const v2f d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u].y, true);
            const float v[8] = {a.x * s[u], a.y * s[u], b.x * s[u], b.y * s[u],
                                c.x * s[u], c.y * s[u], d.x * s[u], d.y * s[u]};
            store_values<OUT_F32>(out, g, v);
        }
    }
}

unsigned grid_for(int64_t lanes) {
    const int64_t b = (lanes + 256 * U - 1) / (256 * U);
    return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

hipError_t launch_mxfp4_quant(const void* x, int in_is_f32, int64_t n_blocks, uint8_t* q, uint8_t* scale,
                              hipStream_t st) {
    const int64_t lanes = n_blocks * 4;
    auto* qw = reinterpret_cast<uint32_t*>(q);
    if (in_is_f32)
        hipLaunchKernelGGL(mxfp4_quant_kernel<true>, dim3(grid_for(lanes)), dim3(256), 0, st, x, lanes, qw, scale);
    else
        hipLaunchKernelGGL(mxfp4_quant_kernel<false>, dim3(grid_for(lanes)), dim3(256), 0, st, x, lanes, qw, scale);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t n_blocks, int out_is_f32, void* out,
                                hipStream_t st) {
    const int64_t lanes = n_blocks * 4;
    const auto* qw = reinterpret_cast<const uint32_t*>(q);
    if (out_is_f32)
        hipLaunchKernelGGL(mxfp4_dequant_kernel<true>, dim3(grid_for(lanes)), dim3(256), 0, st, qw, scale, lanes, out);
    else
        hipLaunchKernelGGL(mxfp4_dequant_kernel<false>, dim3(grid_for(lanes)), dim3(256), 0, st, qw, scale, lanes, out);
    return hipGetLastError();
}

hipError_t launch_fp8_dequant_1x128(const uint8_t* q, const float* scale, int64_t n_tiles, int out_is_f32, void* out,
                                    hipStream_t st) {
    const int64_t lanes = n_tiles * 16;
    const auto* qw = reinterpret_cast<const uint2*>(q);
    if (out_is_f32)
        hipLaunchKernelGGL(fp8_dequant_1x128_kernel<true>, dim3(grid_for(lanes)), dim3(256), 0, st, qw, scale, lanes,
                           out);
    else
        hipLaunchKernelGGL(fp8_dequant_1x128_kernel<false>, dim3(grid_for(lanes)), dim3(256), 0, st, qw, scale, lanes,
                           out);
    return hipGetLastError();
}

}  // namespace moe
