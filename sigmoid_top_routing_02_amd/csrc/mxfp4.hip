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
// All three stream HBM and write what they write once: every access of a wave is
// one contiguous run, at most 16 bytes a lane, and large outputs are stored
// non-temporally (streamed).  On 32768 x 7168 values, bytes read and written: quantised
// from FP32 in 179 us (5.9 TB/s), from bf16 in 98 us (6.1); FP8 to FP32 167 us (7.1),
// to bf16 103 us (6.9); back to FP32 148 us (7.2) and to bf16 86 us (6.9) in a stream
// of such calls alone, to FP32 198 us (5.4) right after a quantisation each.
#include "device_math.h"
#include "kernels.h"
#include "streaming.h"

namespace moe {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// (by value: a vector's element cast in place reads another's bits)
__device__ __forceinline__ v2bf as_bf16x2(uint32_t w) { return __builtin_bit_cast(v2bf, w); }

// The float 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// 8 values a lane, four lanes one block (its maximum is two lane exchanges), U
// steps of the grid in flight per lane: one of FP32's 32 bytes, two of bf16's 16
// (32768 x 7168, NT: FP32 177 us with one and 186 with two, bf16 106 and 95).
template <bool IN_F32, bool NT>
__global__ __launch_bounds__(256) void mxfp4_quant_kernel(const void* __restrict__ x, int64_t lanes,
                                                          uint32_t* __restrict__ q, uint8_t* __restrict__ scale) {
    // `lanes` is a multiple of 4 and so is every stride: the lanes of a block
    // are live together
    constexpr int U = IN_F32 ? 1 : 2;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 + threadIdx.x; g0 - threadIdx.x < lanes; g0 += stride * U) {
        v4u raw[U][IN_F32 ? 2 : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            const v4u* p = static_cast<const v4u*>(x) + (g < lanes ? g : 0) * (IN_F32 ? 2 : 1);
            raw[u][0] = IN_F32 || !NT ? p[0] : __builtin_nontemporal_load(p);
            if constexpr (IN_F32) raw[u][1] = p[1];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            uint32_t m;                                  // exponent field of the largest magnitude
            if constexpr (IN_F32) {
                const v4u a = raw[u][0], b = raw[u][1];
                m = umax(umax(umax(a.x << 1, a.y << 1), umax(a.z << 1, a.w << 1)),
                         umax(umax(b.x << 1, b.y << 1), umax(b.z << 1, b.w << 1)));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64)) >> 24;
            } else {
                const v4u a = raw[u][0];
                m = umax(umax(umax(a.x << 17, a.y << 17), umax(a.z << 17, a.w << 17)),
                         umax(umax(a.x & 0x7FFF0000u, a.y & 0x7FFF0000u), umax(a.z & 0x7FFF0000u, a.w & 0x7FFF0000u)) << 1);
                m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
                m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64)) >> 24;
            }
            const uint32_t byte = m == 255u ? 255u : m > 2u ? m - 2u : 0u;
            const float s = e8m0(byte == 255u ? 127u : byte);
            uint32_t w = 0;
            if constexpr (IN_F32) {
                const v4u a = raw[u][0], b = raw[u][1];
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a.x), __uint_as_float(a.y), s, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a.z), __uint_as_float(a.w), s, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b.x), __uint_as_float(b.y), s, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b.z), __uint_as_float(b.w), s, 3);
            } else {
                const v4u a = raw[u][0];
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a.x), s, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a.y), s, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a.z), s, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a.w), s, 3);
            }
            if (g < lanes) {
                put<NT>(q + g, byte == 255u ? 0u : w);
                if ((g & 3) == 0) scale[g >> 2] = (uint8_t)byte;
            }
        }
    }
}

// The 16 bytes that a lane of the dequantisers stores: 4 FP32 or 8 bf16 values.
template <bool OUT_F32>
__device__ __forceinline__ v4u pack_values(const float* v) {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (OUT_F32) {
            w[i] = __float_as_uint(v[i]);
        } else {
            const v2bf b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, b);
        }
    }
    return w;
}

// Exact: an E2M1 value times a power of two is a bf16 and a binary32 value
// (subnormals included), but for 4 and 6 times the scale 2^127, which no
// quantiser output has and which overflow to infinity.  (8 FP32 values a lane, whose
// two 16-byte stores each skip every other 16 bytes, lost: 199 us against 148 in a
// stream of calls on 32768 x 7168 values.)
template <bool OUT_F32, bool NT>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const void* __restrict__ q,
                                                            const uint8_t* __restrict__ scale, int64_t lanes,
                                                            v4u* __restrict__ out) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < lanes; g += stride) {
        const uint32_t w = OUT_F32 ? static_cast<const uint16_t*>(q)[g] : static_cast<const uint32_t*>(q)[g];
        const uint32_t s = scale[g >> (OUT_F32 ? 3 : 2)];
        const float sc = s == 255u ? __builtin_nanf("") : e8m0(s);
        const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        float v[8] = {a.x * sc, a.y * sc, b.x * sc, b.y * sc};
        if constexpr (!OUT_F32) {
            const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
            const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
            v[4] = c.x * sc;
            v[5] = c.y * sc;
            v[6] = d.x * sc;
            v[7] = d.y * sc;
        }
        put<NT>(out + g, pack_values<OUT_F32>(v));
    }
}

// E4M3(q) * scale in binary32, rounded once where the output is bf16.
template <bool OUT_F32, bool NT>
__global__ __launch_bounds__(256) void fp8_dequant_1x128_kernel(const void* __restrict__ q,
                                                                const float* __restrict__ scale, int64_t lanes,
                                                                v4u* __restrict__ out) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < lanes; g += stride) {
        const uint2 w = OUT_F32 ? make_uint2(static_cast<const uint32_t*>(q)[g], 0u) : static_cast<const uint2*>(q)[g];
        const float s = scale[g >> (OUT_F32 ? 5 : 4)];
        const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
        const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
        float v[8] = {a.x * s, a.y * s, b.x * s, b.y * s};
        if constexpr (!OUT_F32) {
            const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
            const v2f d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
            v[4] = c.x * s;
            v[5] = c.y * s;
            v[6] = d.x * s;
            v[7] = d.y * s;
        }
        put<NT>(out + g, pack_values<OUT_F32>(v));
    }
}

unsigned grid_for(int64_t lanes, int per) {
    return launch_blocks((lanes + 256 * per - 1) / (256 * per), 256);
}

}  // namespace

hipError_t launch_mxfp4_quant(const void* x, int in_is_f32, int64_t n_blocks, uint8_t* q, uint8_t* scale,
                              hipStream_t st) {
    const int64_t lanes = n_blocks * 4;
    auto* qw = reinterpret_cast<uint32_t*>(q);
    auto go = [&](auto kernel, int per) {
        hipLaunchKernelGGL(kernel, dim3(grid_for(lanes, per)), dim3(256), 0, st, x, lanes, qw, scale);
        return hipGetLastError();
    };
    if (streamed(n_blocks * 17)) return in_is_f32 ? go(mxfp4_quant_kernel<true, true>, 1) : go(mxfp4_quant_kernel<false, true>, 2);
    return in_is_f32 ? go(mxfp4_quant_kernel<true, false>, 1) : go(mxfp4_quant_kernel<false, false>, 2);
}

hipError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t n_blocks, int out_is_f32, void* out,
                                hipStream_t st) {
    const int64_t lanes = n_blocks * (out_is_f32 ? 8 : 4);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid_for(lanes, 1)), dim3(256), 0, st, (const void*)q, scale, lanes,
                           static_cast<v4u*>(out));
        return hipGetLastError();
    };
    if (streamed(lanes * 16)) return out_is_f32 ? go(mxfp4_dequant_kernel<true, true>) : go(mxfp4_dequant_kernel<false, true>);
    return out_is_f32 ? go(mxfp4_dequant_kernel<true, false>) : go(mxfp4_dequant_kernel<false, false>);
}

hipError_t launch_fp8_dequant_1x128(const uint8_t* q, const float* scale, int64_t n_tiles, int out_is_f32, void* out,
                                    hipStream_t st) {
    const int64_t lanes = n_tiles * (out_is_f32 ? 32 : 16);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid_for(lanes, 1)), dim3(256), 0, st, (const void*)q, scale, lanes,
                           static_cast<v4u*>(out));
        return hipGetLastError();
    };
    if (streamed(lanes * 16)) return out_is_f32 ? go(fp8_dequant_1x128_kernel<true, true>) : go(fp8_dequant_1x128_kernel<false, true>);
    return out_is_f32 ? go(fp8_dequant_1x128_kernel<true, false>) : go(fp8_dequant_1x128_kernel<false, false>);
}

}  // namespace moe
