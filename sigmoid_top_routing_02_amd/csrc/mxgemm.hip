// Product of MXFP4 matrices grouped by expert (and, with one group, the dense
// MXFP4 product):
//     C[m,n] = sum_b 2^(ea[m,b] + eb[n,b]) * sum_{k in block b} a[m,k] b[n,k],
// blocks of 32 along K, E2M1 codes, E8M0 scale bytes.  One scaled matrix
// instruction (16x16x128 on FP4 operands) takes four blocks with their scales
// and accumulates in FP32, so the whole of K is one chain of them.
//
// Which K a lane holds.  The instruction's lane l supplies row l % 16 and the
// 32 values number l / 16 of the slice, 16 bytes, and one scale byte chosen
// from a register at compile time.  A sum does not depend on the order of its
// terms, so the four slices of a 512-value chunk (16 blocks) are dealt out so
// that lane l's four operands are blocks 4 (l / 16) .. + 3: consecutive in the
// row, 64 bytes of codes, and their four scale bytes one aligned word.  Both
// operands are dealt the same way, and rows are read as the quantiser wrote
// them, with no second layout of codes or scales.
//
// The weights are the instruction's first operand: a lane then holds four
// neighbouring columns of one output row.
#include "device_math.h"
#include "kernels.h"
#include "moe_fp8.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Past the end of every descriptor below (the C ABI keeps their sizes at or
// under it), with room for a 16-byte access and its immediate offset under 2^32:
// reads there return 0 and touch no memory.
constexpr uint32_t OUT = 0xFFFF0000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// c += A B over slice J of a chunk: 16 codes' bytes a lane, scale byte J of sa and sb.
template <int J>
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c, uint32_t sa, uint32_t sb) {
    const v8i x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const v8i y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, J, (int)sa, J, (int)sb);
}

// A lane's share of a chunk of one row.
struct Chunk {
    v4u q[4];
    uint32_t s;
};

// Loads blocks 16 c + 4 kb .. + 3 of a row; blocks past the row's end, and rows
// that are none (row offsets OUT), read zero codes under a zero byte, which is
// a scale and no NaN.  KA: K % 128 == 0, so that the four blocks are in the row
// together and the scale word is aligned.
template <bool KA>
__device__ __forceinline__ void load_chunk(Chunk& f, __amdgpu_buffer_rsrc_t q, __amdgpu_buffer_rsrc_t s,
                                           uint32_t row_q, uint32_t row_s, int blk, int nblk) {
    if constexpr (KA) {
        const bool in = blk < nblk && row_q != OUT;
        const uint32_t o = in ? row_q + (uint32_t)blk * 16u : OUT;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.q[j] = __builtin_amdgcn_raw_buffer_load_b128(q, o + 16u * j, 0, 0);
        f.s = __builtin_amdgcn_raw_buffer_load_b32(s, in ? row_s + (uint32_t)blk : OUT, 0, 0);
    } else {
        f.s = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = blk + j < nblk && row_q != OUT;
            f.q[j] = __builtin_amdgcn_raw_buffer_load_b128(q, in ? row_q + (uint32_t)(blk + j) * 16u : OUT, 0, 0);
            f.s |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(s, in ? row_s + (uint32_t)(blk + j) : OUT, 0, 0)
                   << (8 * j);
        }
    }
}

// SiLU with the hardware exp and reciprocal: relative error of a few 2^-23,
// against the 2^-9 (bf16) or 2^-2 (E2M1) of the rounding that follows.
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ __forceinline__ v4f swiglu(v4f gate, v4f up) {
    v4f h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu(gate[i]) * up[i];
    return h;
}

__device__ __forceinline__ uint2 pack4(v4f v) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

// Columns n .. n+3 of row m of an [*, ld] output, FP32 or bf16, cut at ld.
template <bool F32>
__device__ __forceinline__ void store4(void* out, int64_t m, int n, int ld, v4f v) {
    const int64_t at = m * ld + n;
    if ((ld & 3) == 0) {                                  // rows start on 4 elements; n is a multiple of 4
        if (n < ld) {
            if constexpr (F32) *reinterpret_cast<v4f*>(static_cast<float*>(out) + at) = v;
            else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = pack4(v);
        }
    } else {
        const uint2 w = pack4(v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < ld) {
                if constexpr (F32) static_cast<float*>(out)[at + i] = v[i];
                else static_cast<uint16_t*>(out)[at + i] = (uint16_t)((i & 2 ? w.y : w.x) >> (16 * (i & 1)));
            }
    }
}

// 32 columns of h as one MXFP4 block by the quantiser's rule: lane l has columns
// 4 (l / 16) + i (lo) and 16 + 4 (l / 16) + i (hi) of row l % 16.  Every lane of
// the wave takes part; `live` lanes store.
__device__ __forceinline__ void store_mx_block(uint8_t* out_q, uint8_t* out_s, int64_t block, int kb, bool live,
                                               v4f lo, v4f hi) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __float_as_uint(lo[i]) << 1, b = __float_as_uint(hi[i]) << 1;
        m = a > m ? a : m;
        m = b > m ? b : m;
    }
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)m, o, 64);
        m = b > m ? b : m;
    }
    m >>= 24;
    const uint32_t byte = m == 255u ? 255u : m > 2u ? m - 2u : 0u;
    const float s = byte == 255u ? 1.0f : __uint_as_float(byte ? byte << 23 : 0x00400000u);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[0], lo[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[2], lo[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, hi[0], hi[1], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, hi[2], hi[3], s, 3);
    if (byte == 255u) w = 0;
    if (live) {
        uint16_t* o = reinterpret_cast<uint16_t*>(out_q + block * 16);
        o[kb] = (uint16_t)w;
        o[4 + kb] = (uint16_t)(w >> 16);
        if (kb == 0) out_s[block] = (uint8_t)byte;
    }
}

// First row of B behind column tile `tile` (16 columns) of a block that starts
// at output column c0.  SwiGLU blocks have their gate columns in the first half
// of their NT tiles and the matching up columns in the second: h column c comes
// of B rows 256 (c / 128) + c % 128 and 128 further on.
template <int EPI, int NT>
__device__ __forceinline__ int b_row(int c0, int tile) {
    if constexpr (EPI == MOE_MX_STORE_F32 || EPI == MOE_MX_STORE_BF16) {
        return c0 + tile * 16;
    } else {
        const int c = c0 + (tile % (NT / 2)) * 16;
        return (c >> 7) * 256 + (c & 127) + (tile >= NT / 2 ? 128 : 0);
    }
}

// Few rows to a group (decode): bound by the bytes of B, each read once.  A
// block has NT tiles of 16 B rows of one group; its four waves take every fourth
// chunk of K and add up through LDS, so that a single row of a single group
// still fills the card.  B and the rows of A go straight to registers, the next
// chunk's loads under way while this one is multiplied.
template <int EPI, int MI, int NT, bool KA>
__global__ __launch_bounds__(256) void mxgemm_rows_kernel(MxGemmArgs p) {
    constexpr bool SWIGLU = EPI == MOE_MX_SWIGLU_BF16 || EPI == MOE_MX_SWIGLU_QUANT;
    constexpr int COLS = SWIGLU ? NT * 8 : NT * 16;      // output columns of a block
    __shared__ v4f red[4][MI * NT][64];
    const int lane = threadIdx.x & 63, lr = lane & 15, kb = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = blockIdx.y;
    const int total = (int)p.M_total;
    // offsets outside [0, M_total] (which the caller must not pass) are held inside it
    const int lo = min(max(p.group_offset[g], 0), total);
    const int hi = min(p.group_offset[g + 1], total);
    if (lo >= hi) return;
    const int nblk = p.K / 32, nchunk = (nblk + 15) / 16;
    const uint32_t rb = (uint32_t)p.K / 2;               // bytes of a row of codes
    const auto aq = make_rsrc(p.a_q, (uint32_t)(p.a_rows * rb)), as = make_rsrc(p.a_s, (uint32_t)(p.a_rows * nblk));
    const auto bq = make_rsrc(p.b_q + (int64_t)g * p.N * rb, (uint32_t)p.N * rb);
    const auto bs = make_rsrc(p.b_s + (int64_t)g * p.N * nblk, (uint32_t)p.N * (uint32_t)nblk);
    const int c0 = blockIdx.x * COLS;
    uint32_t bro[NT], bso[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t n = (uint32_t)min(b_row<EPI, NT>(c0, t) + lr, p.N - 1);     // columns past N are not stored
        bro[t] = n * rb;
        bso[t] = n * (uint32_t)nblk;
    }
    for (int m0 = lo; m0 < hi; m0 += 16 * MI) {
        uint32_t aro[MI], aso[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = m0 + i * 16 + lr;
            const uint32_t r = m < hi ? (p.a_row_index ? (uint32_t)p.a_row_index[m] : (uint32_t)m) : 0xFFFFFFFFu;
            const bool in = (int64_t)r < p.a_rows;       // a row that A does not have counts as zeros
            aro[i] = in ? r * rb : OUT;
            aso[i] = in ? r * (uint32_t)nblk : OUT;
        }
        v4f acc[NT][MI];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MI; ++i) acc[t][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        Chunk fa[2][MI], fb[2][NT];
        auto load = [&](int buf, int c) {
            const int blk = c * 16 + kb * 4;             // past the last chunk everything reads zero
#pragma unroll
            for (int t = 0; t < NT; ++t) load_chunk<KA>(fb[buf][t], bq, bs, bro[t], bso[t], blk, nblk);
#pragma unroll
            for (int i = 0; i < MI; ++i) load_chunk<KA>(fa[buf][i], aq, as, aro[i], aso[i], blk, nblk);
        };
        auto multiply = [&](int buf) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    acc[t][i] = mfma<0>(fb[buf][t].q[0], fa[buf][i].q[0], acc[t][i], fb[buf][t].s, fa[buf][i].s);
                    acc[t][i] = mfma<1>(fb[buf][t].q[1], fa[buf][i].q[1], acc[t][i], fb[buf][t].s, fa[buf][i].s);
                    acc[t][i] = mfma<2>(fb[buf][t].q[2], fa[buf][i].q[2], acc[t][i], fb[buf][t].s, fa[buf][i].s);
                    acc[t][i] = mfma<3>(fb[buf][t].q[3], fa[buf][i].q[3], acc[t][i], fb[buf][t].s, fa[buf][i].s);
                }
        };
        load(0, wave);
        for (int c = wave; c < nchunk; c += 8) {
            load(1, c + 4);
            multiply(0);
            load(0, c + 8);
            multiply(1);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MI; ++i) red[wave][t * MI + i][lane] = acc[t][i];
        __syncthreads();
        auto sum = [&](int t, int i) {
            v4f s = red[0][t * MI + i][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) s += red[w][t * MI + i][lane];
            return s;
        };
        if constexpr (EPI == MOE_MX_SWIGLU_QUANT) {
            for (int u = wave; u < NT / 4 * MI; u += 4) {          // 32 columns of 16 rows
                const int t = u / MI * 2, i = u % MI, m = m0 + i * 16 + lr;
                const v4f a = swiglu(sum(t, i), sum(t + NT / 2, i));
                const v4f b = swiglu(sum(t + 1, i), sum(t + 1 + NT / 2, i));
                store_mx_block(p.out_q, p.out_s, (int64_t)m * (p.N / 64) + (c0 + t * 16) / 32, kb, m < hi, a, b);
            }
        } else if constexpr (SWIGLU) {
            for (int u = wave; u < NT / 2 * MI; u += 4) {
                const int t = u / MI, i = u % MI, m = m0 + i * 16 + lr;
                const v4f h = swiglu(sum(t, i), sum(t + NT / 2, i));
                if (m < hi) store4<false>(p.out, m, c0 + t * 16 + kb * 4, p.N / 2, h);
            }
        } else {
            for (int u = wave; u < NT * MI; u += 4) {
                const int t = u / MI, i = u % MI, m = m0 + i * 16 + lr;
                const v4f v = sum(t, i);
                if (m < hi) store4<EPI == MOE_MX_STORE_F32>(p.out, m, c0 + t * 16 + kb * 4, p.N, v);
            }
        }
        __syncthreads();
    }
}

template <int EPI, int MI>
void launch_rows(const MxGemmArgs& a, hipStream_t st) {
    constexpr int NT = 4;
    constexpr int COLS = EPI == MOE_MX_SWIGLU_BF16 || EPI == MOE_MX_SWIGLU_QUANT ? NT * 8 : NT * 16;
    const int cols = EPI == MOE_MX_SWIGLU_BF16 || EPI == MOE_MX_SWIGLU_QUANT ? a.N / 2 : a.N;
    const dim3 grid((cols + COLS - 1) / COLS, a.G);
    if (a.K % 128 == 0)
        hipLaunchKernelGGL((mxgemm_rows_kernel<EPI, MI, NT, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((mxgemm_rows_kernel<EPI, MI, NT, false>), grid, dim3(256), 0, st, a);
}

template <int EPI>
void launch_epi(const MxGemmArgs& a, hipStream_t st) {
    const int64_t rows = (a.M_total + a.G - 1) / a.G;    // rows of a group, on the average
    if (rows <= 16) launch_rows<EPI, 1>(a, st);
    else launch_rows<EPI, 4>(a, st);
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(const MxGemmArgs& a, int epi, hipStream_t st) {
    switch (epi) {
        case MOE_MX_STORE_F32: launch_epi<MOE_MX_STORE_F32>(a, st); break;
        case MOE_MX_STORE_BF16: launch_epi<MOE_MX_STORE_BF16>(a, st); break;
        case MOE_MX_SWIGLU_BF16: launch_epi<MOE_MX_SWIGLU_BF16>(a, st); break;
        default: launch_epi<MOE_MX_SWIGLU_QUANT>(a, st); break;
    }
    return hipGetLastError();
}

}  // namespace moe
