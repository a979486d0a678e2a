// Product of MXFP4 matrices grouped by expert (and, with one group, the dense
// MXFP4 product):
//     C[m,n] = sum_b 2^(ea[m,b] + eb[n,b]) * sum_{k in block b} a[m,k] b[n,k],
// blocks of 32 along K, E2M1 codes, E8M0 scale bytes.  One scaled matrix
// instruction on FP4 operands takes four blocks of 16 rows (16x16x128, the few-row
// kernel) or two of 32 (32x32x64, the tiles) with their scales and accumulates in
// FP32, so the whole of K is one chain of them.
//
// A lane of the instruction supplies one row, 32 consecutive values of it (16
// bytes) and one scale byte, chosen from a register at compile time.  Rows of codes
// and scales are read as the quantiser wrote them: there is no second layout of
// either.
//
// The weights are the instruction's first operand: a lane then holds four
// neighbouring columns of one output row.
#include <atomic>
#include <utility>

#include "device_math.h"
#include "kernels.h"
#include "moe_fp8.h"
#include "mxchoose.h"
#include "mxoffsets.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

#define FENCE() __builtin_amdgcn_sched_barrier(0)

template <int V>
struct IC { static constexpr int value = V; };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// c += A B over 128 values of K: lane l has row l % 16 and block l / 16 of each
// operand, its scale in the low byte.
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c, uint32_t sa, uint32_t sb) {
    const v8i x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const v8i y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// 16 scale bytes of a row, blocks 16 c .. + 15; those past the row's nblk blocks
// are zero, whatever lies there.  KA: the row starts on a word.  Otherwise the
// five words around the bytes are read (the last row's may hold up to three bytes
// past the tensor's end, in the word of its last byte) and shifted.
template <bool KA>
struct Scales {
    v4u w;
    uint32_t more;
    template <bool WHOLE = false>                        // all 16 blocks are in the row
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t d, uint32_t row, int c) {
        const BufferOffset at = scales_of_chunk(KA && WHOLE, KA ? row : row & ~3u, c);
        w = __builtin_amdgcn_raw_buffer_load_b128(d, at.vector, at.scalar, 0);
        if constexpr (!KA) more = __builtin_amdgcn_raw_buffer_load_b32(d, at.vector + 16u, at.scalar, 0);
    }
    template <bool WHOLE = false>
    __device__ __forceinline__ v4u bytes(uint32_t row, int c, int nblk) const {
        v4u v = w;
        if constexpr (!KA) {
            const uint32_t sh = (row & 3u) * 8u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = (uint32_t)((((uint64_t)(j < 3 ? w[j + 1] : more) << 32) | w[j]) >> sh);
        }
        if constexpr (WHOLE) return v;
        const int left = nblk - c * 16;                  // of the row's blocks
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = left - 4 * j;
            v[j] = n >= 4 ? v[j] : n <= 0 ? 0u : KA ? v[j] : v[j] & ((1u << (8 * n)) - 1u);
        }
        return v;
    }
};

// SiLU with the hardware exp and reciprocal: relative error of about (16 + |z|) 2^-23,
// the rounding of the exponential's argument included, against the 2^-9 (bf16) or
// 2^-2 (E2M1) of the rounding that follows.  From z = -87.3 down, where the reciprocal
// would be subnormal, the result is 0 (SiLU is within 88 2^-126 of that).
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

// 16 bytes of row m of an [*, ld] output from column n on, FP32 or bf16, cut at ld.
template <bool F32>
__device__ __forceinline__ void store16(void* out, int64_t m, int n, int ld, v4u x) {
    constexpr int PER = F32 ? 4 : 8;
    const int64_t at = m * ld + n;
    if (ld % PER == 0) {                                  // rows start on 16 bytes; n is a multiple of PER
        if (n < ld) *reinterpret_cast<v4u*>(static_cast<char*>(out) + at * (16 / PER)) = x;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (n + i < ld) {
                if constexpr (F32) static_cast<uint32_t*>(out)[at + i] = x[i];
                else static_cast<uint16_t*>(out)[at + i] = (uint16_t)(x[i / 2] >> (16 * (i & 1)));
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

// 32 columns of h as one MXFP4 block, lane l having columns 8 q + 4 (l / 32) + e
// of row l % 32 in h[q][e]: the two lanes of a row exchange half their codes and
// store 8 bytes each.
__device__ __forceinline__ void store_mx_row(uint8_t* out_q, uint8_t* out_s, int64_t block, int kb, bool live,
                                             const v4f (&h)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = __float_as_uint(h[q][e]) << 1;
            m = a > m ? a : m;
        }
    const uint32_t o = (uint32_t)__shfl_xor((int)m, 32, 64);
    m = (o > m ? o : m) >> 24;
    const uint32_t byte = m == 255u ? 255u : m > 2u ? m - 2u : 0u;
    const float s = byte == 255u ? 1.0f : __uint_as_float(byte ? byte << 23 : 0x00400000u);
    uint32_t w[2];                                       // 16 bits of codes for each q
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h[2 * i][0], h[2 * i][1], s, 0);
        w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], h[2 * i][2], h[2 * i][3], s, 1);
        w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], h[2 * i + 1][0], h[2 * i + 1][1], s, 2);
        w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], h[2 * i + 1][2], h[2 * i + 1][3], s, 3);
        if (byte == 255u) w[i] = 0;
    }
    // bytes of the block: q = 0 lanes' 2, their partners' 2, q = 1, ...; lane 0 of
    // a row keeps q = 0 and 1, its partner q = 2 and 3
    const uint32_t mine = kb ? w[1] : w[0], got = (uint32_t)__shfl_xor((int)(kb ? w[0] : w[1]), 32, 64);
    const uint32_t lo = kb ? got : mine, hi = kb ? mine : got;
    if (live) {
        *reinterpret_cast<uint2*>(out_q + block * 16 + kb * 8) =
            make_uint2((lo & 0xFFFFu) | (hi << 16), (lo >> 16) | (hi & 0xFFFF0000u));
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

// ---------------------------------------------------------------- few rows to a group
//
// Decoding: bound by the bytes of B, each read once.  A block has NT tiles of 16 B
// rows of one group; its four waves take every fourth chunk of 512 values of K and
// add up through LDS, so that a single row of a few groups still fills the card.
// Operands go straight to registers, one access taking 64 consecutive bytes of each
// of 16 rows.  Lane l takes block 4 j + l / 16 of a chunk in its slice j, and byte
// l / 16 of the chunk's scale word j.  A wave sends for a whole chunk of all its
// tiles before it uses any (left to itself the compiler mixes the two, to save
// registers: 105 us where this took 93, at 256 rows in 32 groups, N = 4096, K =
// 7168), A first and each line's two halves right after each other (89.7 us, 5.6
// TB/s; in the compiler's order 91 to 95); the next chunk is left to the CU's other
// waves (two chunks in turn in one wave: 112 us).
template <bool KA>
struct Chunk {
    v4u q[4];
    Scales<KA> s;
    // row_q: the lane's first byte of the row's codes, row_s: the row's first scale,
    // or OUT for no row.  WHOLE: all of the chunk's blocks are in the row; otherwise
    // those past its end read zero codes, and bytes() clears their scales.
    template <bool WHOLE>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t dq, __amdgpu_buffer_rsrc_t ds, uint32_t row_q,
                                         uint32_t row_s, int c, int kb, int nblk) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const BufferOffset at = code_of_chunk(WHOLE || c * 16 + j * 4 + kb < nblk, row_q, c, j);
            q[j] = __builtin_amdgcn_raw_buffer_load_b128(dq, at.vector, at.scalar, 0);
            FENCE();                                     // the two halves of a 128-byte line right after each other
        }
        s.template load<WHOLE>(ds, row_s, c);
    }
};

// First row and number of rows of group g (none past the last group).  Offsets
// outside [0, M_total], which the caller must not pass, are held inside it.
__device__ __forceinline__ int2 rows_of(const MxGemmArgs& p, int g, int total) {
    if (g >= p.G) return make_int2(0, 0);
    const int lo = min(max(p.group_offset[g], 0), total), hi = min(max(p.group_offset[g + 1], 0), total);
    return make_int2(lo, max(hi - lo, 0));
}

// The few-row kernel's tile of T rows for grid row y: rows m0 to `end` of group g
// (the tile may end before), none where m0 >= end.  With a row for each group on the
// average, grid row y < G has the first tile of group y, and row G - 1 + s the tile,
// not the first of its group, that starts in rows s T to s T + T - 1 of all: there
// is one at most.  With fewer rows, grid row y has the tile that starts at row y;
// blocks of the empty groups, though they end at once, would leave the others
// unevenly dealt to the CUs (8 rows in 8 of 32 groups, N = 4096, K = 7168: 24.1 us
// against 27.5; in 7 of 256 groups, K = 2048: 8.0 against 11.8; but 64 rows of 256
// groups, N = 1024, K = 2048: 15.2 against 13.6).  Every wave looks for itself.
struct RowTile { int g, m0, end; };

template <int T>
__device__ __forceinline__ RowTile find_tile(const MxGemmArgs& p, int y) {
    const int total = (int)p.M_total, lane = threadIdx.x & 63;
    const bool firsts = total >= p.G;
    if (firsts && y < p.G) {
        const int2 r = rows_of(p, y, total);
        return {y, r.x, r.x + r.y};
    }
    const int slot = firsts ? (y - p.G + 1) * T : y;
    for (int base = 0; base < p.G; base += 256) {
        int at[4], end[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int2 r = rows_of(p, base + i * 64 + lane, total);
            at[i] = r.x + max((slot - r.x + T - 1) & -T, firsts ? T : 0);
            end[i] = r.x + r.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t hit = __ballot(at[i] < end[i] && at[i] < slot + (firsts ? T : 1));
            if (hit) {
                const int l = __builtin_ctzll(hit);
                return {base + i * 64 + l, __builtin_amdgcn_readlane(at[i], l), __builtin_amdgcn_readlane(end[i], l)};
            }
        }
    }
    return {0, 0, 0};
}

// Sum of v over the block's threads before this one (256 threads; wsum: four ints
// of LDS that nothing else uses before the next barrier after the call).
__device__ __forceinline__ int scan_threads(int v, int* wsum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(incl, o, 64);
        if (lane >= o) incl += u;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int at = incl - v;
    for (int w = 0; w < wave; ++w) at += wsum[w];
    return at;
}

template <int EPI, int MI, int NT, bool KA>
__global__ __launch_bounds__(256) void mxgemm_rows_kernel(MxGemmArgs p) {
    constexpr bool SWIGLU = EPI == MOE_MX_SWIGLU_BF16 || EPI == MOE_MX_SWIGLU_QUANT;
    constexpr int COLS = SWIGLU ? NT * 8 : NT * 16;      // output columns of the block
    __shared__ v4f red[4][MI * NT][64];
    const int lane = threadIdx.x & 63, lr = lane & 15, kb = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const RowTile tile = find_tile<16 * MI>(p, blockIdx.y);
    const int g = __builtin_amdgcn_readfirstlane(tile.g), m0 = __builtin_amdgcn_readfirstlane(tile.m0);
    const int hi = __builtin_amdgcn_readfirstlane(tile.end);
    if (m0 >= hi) return;
    const int nblk = p.K / 32, nchunk = (nblk + 15) / 16;
    const uint32_t rb = (uint32_t)p.K / 2;               // bytes of a row of codes
    // Scale descriptors end on a word.  A group's scales may start off one: the
    // descriptor then starts at the word before and the offsets begin at the rest.
    const auto aq = make_rsrc(p.a_q, code_records(p.a_rows, rb));
    const auto as = make_rsrc(p.a_s, scale_records(p.a_rows, nblk, 0u));
    const auto bq = make_rsrc(p.b_q + (int64_t)g * p.N * rb, code_records(p.N, rb));
    const int64_t sg = (int64_t)g * p.N * nblk;
    const uint32_t off = KA ? 0u : (uint32_t)sg & 3u;
    const auto bs = make_rsrc(p.b_s + (sg - off), scale_records(p.N, nblk, off));
    const int c0 = (int)blockIdx.x * COLS;
    uint32_t bro[NT], bso[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t n = (uint32_t)min(b_row<EPI, NT>(c0, t) + lr, p.N - 1);     // columns past N are not stored
        bro[t] = n * rb + (uint32_t)kb * 16u;
        bso[t] = n * (uint32_t)nblk + off;
    }
    uint32_t aro[MI], aso[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = m0 + i * 16 + lr;
        const uint32_t r = m < hi ? (p.a_row_index ? (uint32_t)p.a_row_index[m] : (uint32_t)m) : 0xFFFFFFFFu;
        const bool in = r < (uint32_t)p.a_rows;      // a row that A does not have counts as zeros
        aro[i] = in ? r * rb + (uint32_t)kb * 16u : OUT;
        aso[i] = in ? r * (uint32_t)nblk : OUT;
    }
    v4f acc[NT][MI];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[t][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    Chunk<KA> fa[MI], fb[NT];
    auto load = [&](auto whole, int c) {
        constexpr bool W = decltype(whole)::value;
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i].template load<W>(aq, as, aro[i], aso[i], c, kb, nblk);
#pragma unroll
        for (int t = 0; t < NT; ++t) fb[t].template load<W>(bq, bs, bro[t], bso[t], c, kb, nblk);
        FENCE();                                         // all of them are sent for before any is used
    };
    auto multiply = [&](auto whole, int c) {
        constexpr bool W = decltype(whole)::value;
        v4u sa[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = fa[i].s.template bytes<W>(aso[i], c, nblk);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const v4u sb = fb[t].s.template bytes<W>(bso[t], c, nblk);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    acc[t][i] = mfma16(fb[t].q[j], fa[i].q[j], acc[t][i], sb[j] >> (8 * kb), sa[i][j] >> (8 * kb));
        }
        FENCE();
    };
    constexpr IC<1> whole{};
    constexpr IC<0> part{};
    const int n_whole = nblk / 16;                       // chunks that K fills; what it leaves comes last
    for (int c = wave; c < n_whole; c += 4) {
        load(whole, c);
        multiply(whole, c);
    }
    if (n_whole < nchunk && n_whole % 4 == wave) {
        load(part, n_whole);
        multiply(part, n_whole);
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
    // the waves take the units of output in turn
    if constexpr (EPI == MOE_MX_SWIGLU_QUANT) {
#pragma unroll
        for (int u = 0; u < NT / 4 * MI; ++u) {              // 32 columns of 16 rows
            if (u % 4 != wave) continue;
            const int t = u / MI * 2, i = u % MI, m = m0 + i * 16 + lr;
            const v4f a = swiglu(sum(t, i), sum(t + NT / 2, i));
            const v4f b = swiglu(sum(t + 1, i), sum(t + 1 + NT / 2, i));
            store_mx_block(p.out_q, p.out_s, (int64_t)m * (p.N / 64) + (c0 + t * 16) / 32, kb,
                           m < hi && c0 < p.N / 2, a, b);
        }
    } else if constexpr (SWIGLU) {
#pragma unroll
        for (int u = 0; u < NT / 2 * MI; ++u) {
            if (u % 4 != wave) continue;
            const int t = u / MI, i = u % MI, m = m0 + i * 16 + lr;
            const v4f h = swiglu(sum(t, i), sum(t + NT / 2, i));
            if (m < hi) store4<false>(p.out, m, c0 + t * 16 + kb * 4, p.N / 2, h);
        }
    } else {
#pragma unroll
        for (int u = 0; u < NT * MI; ++u) {
            if (u % 4 != wave) continue;
            const int t = u / MI, i = u % MI, m = m0 + i * 16 + lr;
            const v4f v = sum(t, i);
            if (m < hi) store4<EPI == MOE_MX_STORE_F32>(p.out, m, c0 + t * 16 + kb * 4, p.N, v);
        }
    }
}

template <int EPI, MxKernel K>
hipError_t launch_rows(const MxGemmArgs& a, hipStream_t st) {
    constexpr int MI = mx_rows(K).high / 16, NT = mx_rows(K).tiles;
    const MxGrid g = mx_rows_grid(mx_rows(K), a.M_total, a.G, a.N);
    const dim3 grid((unsigned)g.x, (unsigned)g.y);
    if (a.K % 128 == 0)
        hipLaunchKernelGGL((mxgemm_rows_kernel<EPI, MI, NT, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((mxgemm_rows_kernel<EPI, MI, NT, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- many rows to a group
//
// Block tile 256 x 256, one block of four waves to a CU, a wave has 128 x 128 of it
// in 32 x 32 tiles (32x32x64 scaled instructions, which reach a higher rate than
// 16x16x128 on this card's power: 6.7 against 6.3 PFLOP/s from registers with
// random codes).  The accumulators fill the 256 accumulation registers of a wave,
// so one operand byte read from LDS serves 128 multiplications and LDS is read at a
// quarter of its rate.  Half tiles, 128 x 256, take the groups of up to 128 rows
// and, where that ends sooner, the tiles of a last round that would not fill the CUs
// (8192 x 7168 x 16384: 528 us, 541 with whole tiles alone).
//
// Stages of 128 values of K (64-byte rows) go from memory to LDS by DMA through a
// ring of four, sent for three stages ahead.  The scales of a chunk of four stages
// (16 bytes a row) pass through registers into one of two buffers a chunk ahead,
// one row a thread, so that a line of scales is touched once per chunk and not by
// every wave in every stage.  Lane l's two operands of a stage are blocks
// 2 (l / 32) and + 1 of its four: a row's 16 bytes are put into LDS as the 8 of
// lanes 0-31, stage by stage, then the 8 of lanes 32-63.
constexpr int TN = MX_TILE_COLS;
constexpr int STAGE_BYTES = 64;                          // of a row
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// One LDS object per stage (A's rows, B's rows), named at compile time at every
// access, so that the compiler sees that a read of one does not touch the DMA into
// another.  The scales of an even and of an odd chunk (512 rows of 16 bytes each)
// lie behind the first stage, whose DMA has landed wherever they are read: the
// compiler waits for every DMA before a read that it knows to touch none.
constexpr int B_AT = 256 * STAGE_BYTES, SCALE_AT = 2 * B_AT, SCALE_BYTES = 512 * 16;
__shared__ __attribute__((aligned(1024))) char g_s0[SCALE_AT + 2 * SCALE_BYTES];
__shared__ __attribute__((aligned(1024))) char g_s1[2 * B_AT];
__shared__ __attribute__((aligned(1024))) char g_s2[2 * B_AT];
__shared__ __attribute__((aligned(1024))) char g_s3[2 * B_AT];
template <int ST> __device__ __forceinline__ char* stage_buf() {
    if constexpr (ST == 0) return g_s0;
    else if constexpr (ST == 1) return g_s1;
    else if constexpr (ST == 2) return g_s2;
    else return g_s3;
}

// global -> LDS: lane l's 16 bytes, from voff + soff, land at lds + 16 l.
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, char* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}
// Writes 16 bytes to LDS, unseen by the compiler, which would first wait for every
// DMA under way into the object; the barrier that readers pass waits for it.
__device__ __forceinline__ void lds_put(char* lds, v4u v) {
    asm volatile("ds_write_b128 %0, %1" ::"v"((uint32_t)(uintptr_t)(lds_void*)lds), "v"(v) : "memory");
}

// A row's scale bytes 0 .. 15 in the order in which lanes read them.
__device__ __forceinline__ v4u deal_scales(v4u v) {
    const uint32_t LO = 0x05040100u, HI = 0x07060302u;   // bytes 0, 1 (2, 3) of the second word, then of the first
    return v4u{__builtin_amdgcn_perm(v[1], v[0], LO), __builtin_amdgcn_perm(v[3], v[2], LO),
               __builtin_amdgcn_perm(v[1], v[0], HI), __builtin_amdgcn_perm(v[3], v[2], HI)};
}

// The 16-byte chunk c of row r lies in slot c ^ swz(r) of its 64 bytes: 8
// neighbouring rows read one chunk from 8 slots of 128 bytes, 16 rows from all
// 64 banks.
__device__ __forceinline__ int swz(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }

#define SCHED(KIND, N) __builtin_amdgcn_sched_group_barrier(KIND, N, 0)
constexpr int MFMA = 0x8, VMEM = 0x20, DS_READ = 0x100;

// Elements 4 q .. 4 q + 3 of an accumulator, read where this stands.  (Left to the
// compiler, all 256 copies are made at the end of the loop over K, and spill.)
__device__ __forceinline__ v4f quad(const v16f& x, int q) {
    v4f v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float f;
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(f) : "a"(x[4 * q + e]));
        v[e] = f;
    }
    return v;
}

template <int READS, int LOADS, int... I>
__device__ __forceinline__ void interleave_slots(std::integer_sequence<int, I...>) {
    constexpr int S = sizeof...(I);
    // slot I's share of n things dealt to S slots, the first ones first
#define SHARE(n) (((I + 1) * (n) + S - 1) / S - (I * (n) + S - 1) / S)
    ((SHARE(READS) ? SCHED(DS_READ, SHARE(READS)) : void(), SCHED(MFMA, 1),
      SHARE(LOADS) ? SCHED(VMEM, SHARE(LOADS)) : void()), ...);
#undef SHARE
}

// Deals the LDS reads and vector loads of a step out among its matrix instructions.
template <int MATRIX, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
    interleave_slots<READS, LOADS>(std::make_integer_sequence<int, MATRIX>{});
}

template <int J>
__device__ __forceinline__ v16f mfma32(v4u a, v4u b, v16f c, uint32_t sa, uint32_t sb) {
    const v8i x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const v8i y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, J, (int)sa, J, (int)sb);
}

// First B row, inside the block's 256, of the wave's column tile t (of 4).
template <bool SWIGLU>
__device__ __forceinline__ int tile_row(int wn, int t) {
    return SWIGLU ? wn * 64 + (t & 1) * 32 + (t >> 1) * 128 : wn * 128 + t * 32;
}

// Row tiles of all groups, in LDS: the number of tiles of 256 and of half tiles
// before each group, and each group's first row (and the last one's end).
struct TileLists {
    int full[1025], half[1025], rows[1025];
    int found;
};

// The tiles t, t + t_step, .. < t_end of the list of height BM (256 or 128).
template <int EPI, int BM, bool KA>
__device__ __forceinline__ void run_tiles(const MxGemmArgs& p, TileLists& lists, int t, int t_end, int t_step) {
    constexpr bool SWIGLU = EPI == MOE_MX_SWIGLU_BF16 || EPI == MOE_MX_SWIGLU_QUANT;
    constexpr int MT = BM / 64;                          // 32-row tiles of a wave
    constexpr int A_DMA = BM / 64, B_DMA = TN / 64;      // 1 KiB (16 rows) DMAs of a wave per stage
    constexpr int ND = A_DMA + B_DMA, NSC = KA ? 2 : 4;  // vector loads of a stage, and of a chunk's scales
    constexpr int CHUNK_M = 2048 / BM;                   // row tiles that go through the columns together
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
    const int lr = lane & 31, kb = lane >> 5;
    const int nblk = p.K / 32, nchunk = (nblk + 15) / 16;
    const int n_tiles = (p.N + TN - 1) / TN;
    const uint32_t rb = (uint32_t)p.K / 2;
    const int* start = BM == 256 ? lists.full : lists.half;

    // Scale descriptors end on a word.  A group's scales may start off one: the
    // descriptor then starts at the word before and the offsets begin at the rest.
    const auto aq = make_rsrc(p.a_q, code_records(p.a_rows, rb));
    const auto as = make_rsrc(p.a_s, scale_records(p.a_rows, nblk, 0u));
    auto bq = aq, bs = as;
    struct Tile { int g, m0, hi, n0; } T{}, U{}, V{};   // the tile at work, the one before, the next
    uint32_t aro[A_DMA], bro[B_DMA], aso, bso;
    uint32_t sa[2][MT], sb[2][4];
    Scales<KA> ca, cb;
    v16f acc[4][MT];
    v4u fa[2][MT], fb[2][4];

    // A barrier for LDS alone, which leaves stores and loads under way.
    auto lds_barrier = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    auto locate = [&](int at) {                          // every thread of the block
        lds_barrier();
        const int rt = at / n_tiles;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = tid * 4 + i;
            if (start[g] <= rt && rt < start[g + 1]) lists.found = g;
        }
        lds_barrier();
        Tile v;
        v.g = __builtin_amdgcn_readfirstlane(lists.found);
        const int first = __builtin_amdgcn_readfirstlane(start[v.g]);
        const int n = __builtin_amdgcn_readfirstlane(start[v.g + 1]) - first;    // the group's row tiles
        const int inside = at - first * n_tiles;
        const int chunk = inside / (CHUNK_M * n_tiles), left = inside - chunk * CHUNK_M * n_tiles;
        const int cm = min(CHUNK_M, n - chunk * CHUNK_M);
        v.hi = __builtin_amdgcn_readfirstlane(lists.rows[v.g + 1]);
        v.m0 = __builtin_amdgcn_readfirstlane(lists.rows[v.g]) + (chunk * CHUNK_M + left % cm) * BM;
        if constexpr (BM == 128)                         // the half tiles come after the whole ones
            v.m0 += __builtin_amdgcn_readfirstlane(lists.full[v.g + 1] - lists.full[v.g]) * 256;
        v.n0 = left / cm * TN;
        return v;
    };
    // A 1 KiB DMA fills 16 rows: lane l brings slot l % 4 of row l / 4.
    const int chunk_of = (lane & 3) ^ swz(lane >> 2);
    // Entry i (of A_DMA + 1) of the rows of A that this thread's DMAs and scales need
    // of a tile; find_rows loads them and nothing uses them before the next setup.
    uint32_t am[A_DMA + 1];
    auto row_of = [&](int i) { return i < A_DMA ? (wave * A_DMA + i) * 16 + (lane >> 2) : tid; };
    auto find_rows = [&](const Tile& v) {
#pragma unroll
        for (int i = 0; i <= A_DMA; ++i) {
            const int m = min(v.m0 + row_of(i), v.hi - 1);
            am[i] = p.a_row_index ? (uint32_t)p.a_row_index[m] : (uint32_t)m;
        }
    };
    auto setup = [&](const Tile& v) {
        bq = make_rsrc(p.b_q + (int64_t)v.g * p.N * rb, code_records(p.N, rb));
        const int64_t sg = (int64_t)v.g * p.N * nblk;
        const uint32_t off = KA ? 0u : (uint32_t)sg & 3u;
        bs = make_rsrc(p.b_s + (sg - off), scale_records(p.N, nblk, off));
        auto has = [&](int i) {                          // a row of the tile, and of A
            return row_of(i) < BM && v.m0 + row_of(i) < v.hi && am[i] < (uint32_t)p.a_rows;
        };
#pragma unroll
        for (int i = 0; i < A_DMA; ++i) aro[i] = has(i) ? am[i] * rb + (uint32_t)chunk_of * 16u : OUT;
        aso = has(A_DMA) ? am[A_DMA] * (uint32_t)nblk : OUT;
        // rows past N lie past the end of B's descriptors
#pragma unroll
        for (int i = 0; i < B_DMA; ++i)
            bro[i] = (uint32_t)(v.n0 + (wave * B_DMA + i) * 16 + (lane >> 2)) * rb + (uint32_t)chunk_of * 16u;
        bso = (uint32_t)(v.n0 + tid) * (uint32_t)nblk + off;
    };
    // Stage s of K into LDS stage ST, A and B.  Blocks past the end of K read zero.
    auto send_a = [&](auto stc, int s) {
        constexpr int ST = decltype(stc)::value;
#pragma unroll
        for (int i = 0; i < A_DMA; ++i) {
            const BufferOffset at = code_of_stage(aro[i], s, chunk_of, nblk);
            lds_dma16(aq, at.vector, at.scalar, stage_buf<ST>() + (wave * A_DMA + i) * 1024);
        }
    };
    auto send_b = [&](auto stc, int s) {
        constexpr int ST = decltype(stc)::value;
#pragma unroll
        for (int i = 0; i < B_DMA; ++i) {
            const BufferOffset at = code_of_stage(bro[i], s, chunk_of, nblk);
            lds_dma16(bq, at.vector, at.scalar, stage_buf<ST>() + B_AT + (wave * B_DMA + i) * 1024);
        }
    };
    auto load_scales = [&](int c) {
        ca.load(as, aso, c);
        cb.load(bs, bso, c);
    };
    auto write_scales = [&](int c) {
        char* to = g_s0 + SCALE_AT + (c & 1) * SCALE_BYTES + tid * 16;
        const v4u a = deal_scales(ca.bytes(aso, c, nblk)), b = deal_scales(cb.bytes(bso, c, nblk));
        lds_put(to, a);                                  // of a half tile, 128 rows of zeros that nothing reads
        lds_put(to + 256 * 16, b);
    };
    uint32_t slot[2];                                    // the lane's chunk of step j in its row
#pragma unroll
    for (int j = 0; j < 2; ++j) slot[j] = (uint32_t)(lr * STAGE_BYTES + ((kb * 2 + j) ^ swz(lr)) * 16);
    auto read = [&](auto stc, auto jc) {                 // the operands of step J of stage ST, into set J
        constexpr int ST = decltype(stc)::value, J = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            fb[J][i] = *reinterpret_cast<const v4u*>(stage_buf<ST>() + B_AT + tile_row<SWIGLU>(wn, i) * STAGE_BYTES + slot[J]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            fa[J][i] = *reinterpret_cast<const v4u*>(stage_buf<ST>() + (wm * (BM / 2) + i * 32) * STAGE_BYTES + slot[J]);
    };
    // Word H of the lane's scales of chunk c: stages 2 H and 2 H + 1, bytes 0 and 1
    // those of the first's steps 0 and 1, bytes 2 and 3 of the second's.
    auto read_scales = [&](auto hc, int c) {
        constexpr int H = decltype(hc)::value;
        int off = SCALE_AT + (c & 1) * SCALE_BYTES + lr * 16 + kb * 8 + H * 4;
        asm volatile("" : "+v"(off));                    // opaque: a read that may touch the stage's DMA
        const char* at = g_s0 + off;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sb[H][i] = *reinterpret_cast<const uint32_t*>(at + (256 + tile_row<SWIGLU>(wn, i)) * 16);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            sa[H][i] = *reinterpret_cast<const uint32_t*>(at + (wm * (BM / 2) + i * 32) * 16);
    };
    auto multiply = [&](auto stc, auto jc) {
        constexpr int ST = decltype(stc)::value, J = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                acc[n][i] = mfma32<(ST & 1) * 2 + J>(fb[J][n], fa[J][i], acc[n][i], sb[ST / 2][n], sa[ST / 2][i]);
    };
    constexpr IC<0> c0{};
    constexpr IC<1> c1{};
    constexpr IC<2> c2{};
    constexpr IC<3> c3{};
    // Lane l has columns 8 q + 4 (l / 32) + e of row l % 32 of each 32 x 32 tile in
    // element 4 q + e.  FP32 and bf16 leave through LDS, 32 rows of 128 bytes at a
    // time (two places in turn, the wave's own in the last stage, which the next
    // tile's first three stages leave alone), so that eight lanes store one whole
    // line; chunk c of a row lies in slot c ^ row % 8.
    auto store = [&](const Tile& v) {
        // the reads of quad() are hidden from the compiler, which counts the wait
        // from the last matrix instruction to a read of its result (at most 19)
        asm volatile("s_nop 15\n\ts_nop 15");
        char* mine = g_s3 + wave * 8192;
        auto put16 = [&](int place, int chunk, v4f x) { *reinterpret_cast<v4f*>(mine + place * 4096 + lr * 128 + ((chunk ^ (lr & 7)) << 4)) = x; };
        auto put8 = [&](int place, int chunk, v4f x) {
            *reinterpret_cast<uint2*>(mine + place * 4096 + lr * 128 + ((chunk ^ (lr & 7)) << 4) + kb * 8) = pack4(x);
        };
        auto flush = [&](int place, int m0, int col, int ld) {      // 32 rows from m0, 128 bytes from column col
            constexpr bool F32 = EPI == MOE_MX_STORE_F32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 8 + (lane >> 3);
                const v4u x = *reinterpret_cast<const v4u*>(mine + place * 4096 + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                if (m0 + r < v.hi) store16<F32>(p.out, m0 + r, col + (lane & 7) * (F32 ? 4 : 8), ld, x);
            }
        };
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m0 = v.m0 + wm * (BM / 2) + i * 32;
            FENCE();                                     // one row of tiles at a time out of the accumulators
            if constexpr (EPI == MOE_MX_STORE_F32) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) put16(n & 1, 2 * q + kb, quad(acc[n][i], q));
                    flush(n & 1, m0, v.n0 + tile_row<false>(wn, n), p.N);
                }
            } else if constexpr (EPI == MOE_MX_STORE_BF16) {
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        put8(n / 2, q, quad(acc[n][i], q));
                        put8(n / 2, 4 + q, quad(acc[n + 1][i], q));
                    }
                    flush(n / 2, m0, v.n0 + tile_row<false>(wn, n), p.N);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    v4f h[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) h[q] = swiglu(quad(acc[n][i], q), quad(acc[n + 2][i], q));
                    if constexpr (EPI == MOE_MX_SWIGLU_BF16) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) put8(i & 1, 4 * n + q, h[q]);
                    } else {
                        const int m = m0 + lr, col = v.n0 / 2 + wn * 64 + n * 32;
                        store_mx_row(p.out_q, p.out_s, (int64_t)m * (p.N / 64) + col / 32, kb, m < v.hi, h);
                    }
                }
                if constexpr (EPI == MOE_MX_SWIGLU_BF16) flush(i & 1, m0, v.n0 / 2 + wn * 64, p.N / 2);
            }
        }
    };
    // Waits until all but the last N of this wave's vector memory operations are
    // done and every wave has come here with its LDS reads and writes done.
    auto landed = [](auto nc) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(nc)::value) : "memory");
    };
    // Stage ST of chunk c, stage s = 4 c + ST of K.  Step 0 sends for B of stage
    // s + 3 and step 1 for A of stage s + 4, into the places of stages s - 1 and s,
    // which every wave had read before the last barrier.  Step 1 begins when stage
    // s + 1 has landed (stages s + 2 and s + 3, and the scales on their way, may be
    // out) and reads its first operands; the next chunk's scales are loaded in step
    // 1 of the chunk's first stage and written in step 1 of its third; each half of
    // them is read when the last stage that used its registers is under way.  Past
    // the end of K the same instructions move zeros, so that the loop has no
    // branches.
    auto stage = [&](auto stc, auto nextc, auto sentc, int c) {
        constexpr int ST = decltype(stc)::value;
        FENCE();
        read(stc, c1);
        send_b(sentc, c * 4 + ST + 3);
        if constexpr (ST == 0) read_scales(c1, c);
        multiply(stc, c0);
        interleave<4 * MT, MT + 4 + (ST == 0 ? (MT + 4) / 2 : 0), B_DMA>();
        FENCE();
        landed(IC<2 * ND + (ST == 1 || ST == 2 ? NSC : 0)>{});
        FENCE();
        read(nextc, c0);
        send_a(stc, c * 4 + ST + 4);
        if constexpr (ST == 0) load_scales(c + 1);
        if constexpr (ST == 2) write_scales(c + 1);
        if constexpr (ST == 3) read_scales(c0, c + 1);
        multiply(stc, c1);
        interleave<4 * MT, MT + 4 + (ST == 3 ? (MT + 4) / 2 : 0), A_DMA + (ST == 0 ? NSC : 0)>();
        FENCE();
    };
    // Each tile's place and rows of A are looked up before the tile ahead of it starts.
    if (t < t_end) {
        T = locate(t);
        find_rows(T);
    }
    for (bool before = false;; before = true) {
        const bool more = t < t_end;
        t += t_step;
        if (more) {                                      // the first three stages travel during the last tile's stores
            setup(T);
            load_scales(0);
            FENCE();
            send_a(c0, 0);
            send_b(c0, 0);
            FENCE();
            send_a(c1, 1);
            send_b(c1, 1);
            FENCE();
            send_a(c2, 2);
            send_b(c2, 2);
            FENCE();
            if (t < t_end) {
                V = locate(t);
                find_rows(V);
            }
        }
        if (before) store(U);
        if (!more) break;
        U = T;
        T = V;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[n][i][e] = 0.0f;
        write_scales(0);
        FENCE();
        landed(IC<2 * ND>{});
        FENCE();
        send_a(c3, 3);
        read(c0, c0);
        read_scales(c0, 0);
        int c = 0;
        do {                                             // K > 0: at least once
            stage(c0, c1, c3, c);
            stage(c1, c2, c0, c);
            stage(c2, c3, c1, c);
            stage(c3, c0, c2, c);
        } while (++c < nchunk);
        landed(IC<0>{});                                 // the zeros past the end of K
    }
}

template <int EPI, bool KA>
__global__ __launch_bounds__(256, 1) void mxgemm_tile_kernel(MxGemmArgs p) {
    __shared__ TileLists lists;
    const int tid = threadIdx.x, total = (int)p.M_total;
    const int nchunk = (p.K / 32 + 15) / 16, n_tiles = (p.N + TN - 1) / TN;
    const int xcd = (int)blockIdx.x & 7, t_step = (int)gridDim.x >> 3, block = (int)blockIdx.x >> 3;
    int n_full, n_half;
    {
        // Four groups a thread: a half tile for up to 128 rows, else whole tiles.  (A
        // half tile for a larger group's rest would run after the whole tiles and read
        // B again: 245 us against 235 at 32 groups of 256 rows on the average.)
        int nf[4], nh[4], sum_f = 0, sum_h = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = tid * 4 + i;
            const int2 r = rows_of(p, g, total);
            nf[i] = r.y > 128 ? (r.y + 255) / 256 : 0;
            nh[i] = r.y > 0 && r.y <= 128;
            if (g < p.G) lists.rows[g] = r.x;
            if (g == p.G - 1) lists.rows[p.G] = r.x + r.y;
            sum_f += nf[i];
            sum_h += nh[i];
        }
        int* scratch = reinterpret_cast<int*>(g_s0);
        int at_f = scan_threads(sum_f, scratch), at_h = scan_threads(sum_h, scratch + 4);
        if (tid == 255) {
            scratch[8] = at_f + sum_f;
            scratch[9] = at_h + sum_h;
        }
        __syncthreads();
        n_full = __builtin_amdgcn_readfirstlane(scratch[8]);
        n_half = __builtin_amdgcn_readfirstlane(scratch[9]);
        // How many whole row tiles, the last ones of the list, to make half tiles of:
        // thread x tries x, and the x whose busiest block is done first is taken.  A
        // tile of c chunks takes 11 + 4.5 c us, a half tile 9 + 3.6 c.
        unsigned long long best = ~0ull;
        if (tid <= n_full) {
            const int f = ((n_full - tid) * n_tiles + 7) / 8, all = f + ((n_half + 2 * tid) * n_tiles + 7) / 8;
            const int at[6] = {0, f % t_step - 1, f % t_step, all % t_step - 1, all % t_step, t_step - 1};
            int64_t most = 0;
#pragma unroll
            for (int i = 0; i < 6; ++i) {                // the load changes at these blocks only
                const int j = max(at[i], 0);
                const int whole = f > j ? (f - 1 - j) / t_step + 1 : 0, tiles = all > j ? (all - 1 - j) / t_step + 1 : 0;
                most = max(most, (int64_t)whole * (110 + 45 * nchunk) + (int64_t)(tiles - whole) * (90 + 36 * nchunk));
            }
            best = (unsigned long long)most << 8 | (unsigned)tid;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const unsigned long long b = __shfl_xor(best, o, 64);
            best = b < best ? b : best;
        }
        auto* least = reinterpret_cast<unsigned long long*>(scratch + 16);
        if ((tid & 63) == 0) least[tid >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) best = least[i] < best ? least[i] : best;
        const int split = __builtin_amdgcn_readfirstlane((int)(best & 255u));
        n_full -= split;
        n_half += 2 * split;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lists.full[tid * 4 + i] = min(at_f, n_full);
            lists.half[tid * 4 + i] = at_h + 2 * max(at_f - n_full, 0);
            at_f += nf[i];
            at_h += nh[i];
        }
        if (tid == 255) {
            lists.full[1024] = n_full;
            lists.half[1024] = n_half;
        }
        __syncthreads();
    }
    // Blocks go to the eight XCDs in turn; each XCD has one stretch of each list and
    // its blocks take neighbouring tiles, which share operands in its L2.  The whole
    // tiles are dealt first and the half tiles go on where those end.
    auto stretch = [&](int n, int& first, int& count) {
        const int share = (n + 7) / 8;
        first = xcd * share;
        count = max(min(share, n - first), 0);
    };
    int f0, nf, h0, nh;
    stretch(n_full * n_tiles, f0, nf);                   // the C ABI keeps these under 2^31
    stretch(n_half * n_tiles, h0, nh);
    run_tiles<EPI, 256, KA>(p, lists, f0 + block, f0 + nf, t_step);
    const int behind = block < nf ? (nf - block + t_step - 1) / t_step * t_step + block - nf : block - nf;
    run_tiles<EPI, 128, KA>(p, lists, h0 + behind, h0 + nh, t_step);
}

// CUs of the current device, asked for once per device (any thread may call; a
// lost race asks again).
hipError_t cu_count(int& cus) {
    static std::atomic<int> known[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    cus = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (cus > 0) return hipSuccess;
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess && dev >= 0 && dev < 64) known[dev].store(cus, std::memory_order_relaxed);
    return e;
}

template <int EPI>
hipError_t launch_tiles(const MxGemmArgs& a, int cus, hipStream_t st) {
    const int64_t most = ((a.M_total + 127) / 128 + a.G) * ((a.N + TN - 1) / TN);
    const int64_t want = most < cus ? most : cus;
    const dim3 grid((unsigned)((want + 7) / 8 * 8));      // the same count on every XCD
    if (a.K % 128 == 0) hipLaunchKernelGGL((mxgemm_tile_kernel<EPI, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((mxgemm_tile_kernel<EPI, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_epi(const MxGemmArgs& a, hipStream_t st) {
    // MXFP4 output has no narrow kernel (its blocks of 32 columns of h need four column
    // tiles) and takes 16 rows, 4 tiles in its place.  Choosing among the other four by
    // their times gives 32 rows, 4 tiles there, which is slower (us, 16 / 32 rows): 1 row
    // of N = 4096, K = 1024 3.8 / 4.1, 8 of 8 groups 6.1 / 6.4, 8 rows in each of 32 groups
    // of N = 4096, K = 512 9.9 / 14.5.
    constexpr MxKernel FEW = EPI == MOE_MX_SWIGLU_QUANT ? ROWS16 : ROWS16_NARROW;
    int cus = 0;
    const hipError_t e = cu_count(cus);
    if (e != hipSuccess) return e;
    switch (mx_choose(a.M_total, a.G, a.N, a.K, cus)) {
        case ROWS16_NARROW: return launch_rows<EPI, FEW>(a, st);
        case ROWS16: return launch_rows<EPI, ROWS16>(a, st);
        case ROWS32: return launch_rows<EPI, ROWS32>(a, st);
        case ROWS64: return launch_rows<EPI, ROWS64>(a, st);
        default: return launch_tiles<EPI>(a, cus, st);
    }
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(const MxGemmArgs& a, int epi, hipStream_t st) {
    switch (epi) {
        case MOE_MX_STORE_F32: return launch_epi<MOE_MX_STORE_F32>(a, st);
        case MOE_MX_STORE_BF16: return launch_epi<MOE_MX_STORE_BF16>(a, st);
        case MOE_MX_SWIGLU_BF16: return launch_epi<MOE_MX_SWIGLU_BF16>(a, st);
        default: return launch_epi<MOE_MX_SWIGLU_QUANT>(a, st);
    }
}

}  // namespace moe
