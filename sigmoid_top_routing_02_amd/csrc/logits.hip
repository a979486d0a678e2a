// The router's backward from a gradient of all its logits, x FP32 [T, E]:
//     du = du_in + x . e      (e = centroids, bf16 [E, d]),
//     de = de_in + x^T . u    (u bf16 [T, d]).
// moe_router_backward takes the gates' gradient, K values a token; what the balance
// loss adds is dense.
//
// x = hi + mid + lo exactly, three bf16 of 8 bits each cut off the 24 of an FP32's
// significand, so three bf16 matrix instructions with FP32 accumulation give every
// product exactly and lose nothing of x: 3 times the multiplications at the bf16
// rate are a fifth of the time of the FP32 instructions.  logits_split_kernel
// writes the three planes once; both products then read them by DMA or 16 bytes a
// lane.  Only products and parts under the smallest normal number are lost (the
// matrix instructions flush them).
//
// Both products contract over the rows of a row-major bf16 matrix (e, u), and de
// over x's rows too: those operands' fragments, 8 values down a column, come out of
// LDS by the transposing 8-byte reads (16 lanes read 4 rows of 16 values and each
// gets a column).  16-byte chunks are permuted in LDS so that the four rows of such
// a read lie on different banks (see swizzle).
#include "device_math.h"
#include "kernels.h"
#include "streaming.h"

namespace moe {
namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int CHUNK = 32;               // tokens that the planes hold together

// The chunk of 16 bytes that chunk c of row r lies at, in rows of `bytes` bytes
// (128, 256 or 512): rows r to r + 3 of one 64-byte column fall on different quarters
// of the 256 bytes that the banks span.
template <int BYTES>
__device__ __forceinline__ int swizzle(int r) {
    return BYTES == 128 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}
// 16 bytes a lane, global -> LDS at lds + 16 lane (lds is wave-uniform); past the
// descriptor's range zeros are written
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, char* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}

// A fragment of 8 values down a column: rows k, k + 1, .. k + 7 of which the lane's
// 16 neighbours read 4 rows at p and 4 at p + rows4 (the bytes of 4 rows).
__device__ __forceinline__ v8bf column8(const char* p, int rows4) {
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(char*)p);
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(char*)(p + rows4));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The three planes of x, [chunk][plane][32 tokens][EP] bf16, each token's 16-byte
// chunks permuted by swizzle<2 EP>; zeros past T and E.
template <int EP>
__global__ __launch_bounds__(256) void logits_split_kernel(const float* __restrict__ x, int64_t T, int E,
                                                           char* __restrict__ planes) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;       // (token, 8 experts)
    const int64_t t = at / (EP / 8);
    const int c = (int)(at % (EP / 8));
    float v[8];
    if (t < T && c * 8 + 8 <= E && E % 4 == 0) {
        const float4* p = reinterpret_cast<const float4*>(x + t * E + c * 8);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = t < T && c * 8 + i < E ? x[t * E + c * 8 + i] : 0.0f;
    }
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // an infinity is its own first part; a NaN stays NaN through the second
        const float hi = __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
        const float r = __builtin_fabsf(v[i]) == __builtin_inff() ? 0.0f : v[i] - hi;
        const float mid = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
        const float lo = r - mid;
        const float part[3] = {lo, mid, hi};
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t b = __float_as_uint(part[p]) >> 16;
            w[p][i / 2] = i % 2 ? w[p][i / 2] | b << 16 : b;
        }
    }
    const int64_t chunk = t / CHUNK;
    const int row = (int)(t % CHUNK);
#pragma unroll
    for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint4*>(planes + ((chunk * 3 + p) * CHUNK + row) * (EP * 2) + (c ^ swizzle<EP * 2>(row)) * 16) =
            make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

struct LogitsDuArgs {
    const char* planes;
    const uint16_t* e;
    int64_t T;
    int d, E, steps;                    // steps of 64 columns that a block takes
    const float* in;
    float* out;
};

template <int V> struct IC { static constexpr int value = V; };

constexpr int DU_STEP = 64;             // columns
__shared__ __attribute__((aligned(1024))) char g_e0[256 * DU_STEP * 2];
__shared__ __attribute__((aligned(1024))) char g_e1[256 * DU_STEP * 2];

// du: a wave holds the fragments of its 32 tokens for all experts in registers and goes
// through the columns, the block's four waves sharing 64 columns' centroids at a time
// in LDS, sent for a step ahead; 32 columns are multiplied, added to du_in and stored at
// a time.  Two blocks share a CU, so that one multiplies while the other waits for
// du_in or for its stores to go out.
template <int EP, bool ADD, bool NT>
__global__ __launch_bounds__(256, 2) void logits_du_kernel(LogitsDuArgs a) {
    constexpr int KS = EP / 16;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i16 = lane & 15, half = lane >> 5;
    const int64_t chunks = (a.T + CHUNK - 1) / CHUNK;
    const int64_t chunk = (int64_t)blockIdx.x * 4 + wave;
    const int64_t t0 = chunk * CHUNK;
    const int rows = t0 < a.T ? (int)(a.T - t0 < CHUNK ? a.T - t0 : CHUNK) : 0;
    const int s0 = blockIdx.y * a.steps, s1 = min(s0 + a.steps, a.d / DU_STEP);

    const auto e_rsrc = make_rsrc(a.e, (uint32_t)a.E * (uint32_t)a.d * 2u);
    const int dr = lane >> 3;                       // DMA: row of 8 and chunk of 8
    const uint32_t dma_off = (uint32_t)(wave * 8 + dr) * (uint32_t)a.d * 2u + (uint32_t)((lane & 7) ^ swizzle<128>(dr)) * 16u;
    auto send = [&](auto st, int s) {               // EP / 32 DMAs
        char* const to = decltype(st)::value ? g_e1 : g_e0;
#pragma unroll
        for (int j = 0; j < EP / 32; ++j)
            lds_dma16(e_rsrc, dma_off, (uint32_t)(j * 32) * (uint32_t)a.d * 2u + (uint32_t)s * (DU_STEP * 2u),
                      to + (j * 4 + wave) * 1024);
    };
    // rows past the last token are out of the descriptors' range
    const uint32_t records = (uint32_t)rows * (uint32_t)a.d * 4u, row4 = (uint32_t)a.d * 4u;
    const auto in_rsrc = make_rsrc(ADD ? a.in + t0 * a.d : a.out, ADD ? records : 0u);
    const auto out_rsrc = make_rsrc(a.out + t0 * a.d, records);
    // result i of 16 of the lane's column lane % 32: row 8 (i / 4) + 4 half + i % 4
    const uint32_t out_off = (uint32_t)(4 * half) * row4 + (uint32_t)(lane & 31) * 4u;
    auto at = [&](int i) { return out_off + (uint32_t)(8 * (i / 4) + i % 4) * row4; };
    send(IC<0>{}, s0);
    v8bf x[3][KS];
    {
        const int t = lane & 31;
        const char* p = a.planes + ((chunk < chunks ? chunk : chunks - 1) * 3 * CHUNK + t) * (EP * 2);
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                x[w][k] = *reinterpret_cast<const v8bf*>(p + w * CHUNK * EP * 2 + ((2 * k + half) ^ swizzle<EP * 2>(t)) * 16);
    }
    // the lane's part of a transposing read: row i16 / 4 of 4, 8 bytes of its column;
    // the second 32 columns start 64 bytes on
    const int read_off = (8 * (g >> 1) + (i16 >> 2)) * 128 +
                         ((2 * (g & 1) + ((i16 & 3) >> 1)) ^ swizzle<128>(i16 >> 2)) * 16 + (i16 & 1) * 8;
    auto columns32 = [&](const char* b, int col) {  // col: the first of them
        float old[16];
        if constexpr (ADD) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                old[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in_rsrc, at(i), col * 4, NT ? 2 : 0));
        }
        v8bf f[2];
        f[0] = column8(b, 512);
        v16f acc = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            if (k + 1 < KS) f[(k + 1) & 1] = column8(b + (k + 1) * 2048, 512);   // a round of products ahead
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int w = 0; w < 3; ++w) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[w][k], f[k & 1], acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float o = ADD ? old[i] + acc[i] : acc[i];
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), out_rsrc, at(i), col * 4, NT ? 2 : 0);
        }
    };
    auto step = [&](auto st, int s) {
        constexpr int ST = decltype(st)::value;
        if (s + 1 < s1) send(IC<1 - ST>{}, s + 1);
        __builtin_amdgcn_sched_barrier(0);          // before the stores that the wait below leaves out
        const char* const b = ST ? g_e1 : g_e0;
        columns32(b + read_off, s * DU_STEP);
        columns32(b + (read_off ^ 64), s * DU_STEP + 32);
        // the next stage has landed (32 stores at least were sent for after it: as many may be out) and
        // this one is read
        asm volatile("s_waitcnt vmcnt(32) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    for (int s = s0; s < s1; s += 2) {
        step(IC<0>{}, s);
        if (s + 1 < s1) step(IC<1>{}, s + 1);
    }
}

struct LogitsDeArgs {
    const char* planes;
    const uint16_t* u;
    int64_t T;
    int d, E, chunks;                   // chunks of 32 tokens that a block takes
    float* part;                        // [blockIdx.y][E][d]
};

// The stages are separate LDS objects, so that the compiler sees that reads of one do
// not wait for the DMA into another.
__shared__ __attribute__((aligned(1024))) char g_stage0[64 * 1024];
__shared__ __attribute__((aligned(1024))) char g_stage1[64 * 1024];

template <int ST>
__device__ __forceinline__ char* stage() {
    if constexpr (ST == 0) return g_stage0;
    else return g_stage1;
}

// de: a block takes all experts (EP = 64 WE) by 256 columns over some of the tokens, a
// wave 64 experts by 32 WE columns; x's planes and u's rows come by DMA 32 tokens at
// a time into two stages.
template <int WE>
__global__ __launch_bounds__(512, 2) void logits_de_kernel(LogitsDeArgs a) {
    constexpr int EP = 64 * WE, A_BYTES = 3 * CHUNK * EP * 2, NT = WE;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int we = wave % WE, wn = wave / WE;
    const int g = lane >> 4, i16 = lane & 15;
    const int n0 = blockIdx.x * 256;
    const int64_t chunks = (a.T + CHUNK - 1) / CHUNK;
    const int64_t c0 = (int64_t)blockIdx.y * a.chunks, c1 = c0 + a.chunks < chunks ? c0 + a.chunks : chunks;

    auto send = [&](auto st, int64_t c) {
        char* const to = stage<decltype(st)::value>();
        const auto x_rsrc = make_rsrc(a.planes + c * A_BYTES, A_BYTES);
#pragma unroll
        for (int j = 0; j < (A_BYTES / 1024 + 7) / 8; ++j) {
            const int k = j * 8 + wave;
            if (k < A_BYTES / 1024) lds_dma16(x_rsrc, (uint32_t)lane * 16u, (uint32_t)k * 1024u, to + k * 1024);
        }
        const int64_t t0 = c * CHUNK;
        const int rows = (int)(a.T - t0 < CHUNK ? a.T - t0 : CHUNK);
        const auto u_rsrc = make_rsrc(a.u + t0 * a.d, (uint32_t)rows * (uint32_t)a.d * 2u);
#pragma unroll
        for (int j = 0; j < 2; ++j) {                // two rows of 512 bytes a time; rows past T are out of range
            const int k = j * 8 + wave, r = 2 * k + (lane >> 5);
            const int at = ((lane & 31) ^ swizzle<512>(r)) * 16 + n0 * 2;
            // columns past d: the row's own last ones, whose results are not stored
            lds_dma16(u_rsrc, (uint32_t)r * (uint32_t)a.d * 2u + (uint32_t)min(at, a.d * 2 - 16), 0u, to + A_BYTES + k * 1024);
        }
    };
    v16f acc[2][NT] = {};
    const int row = 8 * (g >> 1) + (i16 >> 2), in16 = 2 * (g & 1) + ((i16 & 3) >> 1);
    const int a_off = row * EP * 2 + ((we * 8 + in16) ^ swizzle<EP * 2>(i16 >> 2)) * 16 + (i16 & 1) * 8;
    const int b_off = A_BYTES + row * 512 + ((wn * NT * 4 + in16) ^ swizzle<512>(i16 >> 2)) * 16 + (i16 & 1) * 8;
    struct Fragments { v8bf x[3][2], b[NT]; };
    auto read = [&](auto st, int k, Fragments& f) {  // 16 tokens of the chunk's 32
        const char* const s = stage<decltype(st)::value>();
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
                f.x[w][m] = column8(s + (a_off ^ (m * 64)) + (w * CHUNK + k * 16) * EP * 2, 4 * EP * 2);
#pragma unroll
        for (int n = 0; n < NT; ++n) f.b[n] = column8(s + (b_off ^ (n * 64)) + k * 16 * 512, 4 * 512);
    };
    auto multiply = [&](const Fragments& f) {
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.x[w][m], f.b[n], acc[m][n], 0, 0, 0);
    };
    // Reads run half a chunk ahead of the products: the second half's while the first
    // half is multiplied, the next chunk's first half's, behind the wait for its DMA,
    // while the second half is.
    Fragments f0, f1;
    auto step = [&](auto st, int64_t c) {
        constexpr int ST = decltype(st)::value;
        read(st, 1, f1);
        multiply(f0);
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (c + 2 < c1) send(st, c + 2);
        if (c + 1 < c1) read(IC<1 - ST>{}, 0, f0);
        multiply(f1);
    };
    send(IC<0>{}, c0);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    if (c0 + 1 < c1) send(IC<1>{}, c0 + 1);
    read(IC<0>{}, 0, f0);
    for (int64_t c = c0; c < c1; c += 2) {
        step(IC<0>{}, c);
        if (c + 1 < c1) step(IC<1>{}, c + 1);
    }
    float* const part = a.part + (int64_t)blockIdx.y * a.E * a.d;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = we * 64 + m * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
                const int col = n0 + (wn * NT + n) * 32 + (lane & 31);
                if (e < a.E && col < a.d) part[(int64_t)e * a.d + col] = acc[m][n][i];
            }
}

// de = de_in + the parts in order; n = E d values, a multiple of 4
__global__ __launch_bounds__(256) void logits_sum_kernel(const float* __restrict__ part, int parts, int64_t n,
                                                         const float* in, float* out) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= n) return;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < parts; ++p) s += *reinterpret_cast<const v4f*>(part + p * n + at);
    if (in) s += *reinterpret_cast<const v4f*>(in + at);
    *reinterpret_cast<v4f*>(out + at) = s;
}

int padded_experts(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : 256; }

int64_t token_chunks(int64_t T) { return (T + CHUNK - 1) / CHUNK; }

size_t plane_bytes(int64_t T, int E) { return (size_t)token_chunks(T) * 3 * CHUNK * padded_experts(E) * 2; }

// Chunks that a block of logits_de_kernel takes.
int de_chunks(int64_t T, int d) {
    const int64_t blocks = (d + 255) / 256, chunks = token_chunks(T), parts = 256 / blocks < 1 ? 1 : 256 / blocks;
    const int64_t each = (chunks + parts - 1) / parts;
    return (int)(each < 4 ? 4 : each);
}

int de_parts(int64_t T, int d) { return (int)((token_chunks(T) + de_chunks(T, d) - 1) / de_chunks(T, d)); }

template <int EP>
void split_and_du(const float* x, const uint16_t* e, int64_t T, int d, int E, const float* in, float* out, char* planes,
                  hipStream_t st) {
    hipLaunchKernelGGL((logits_split_kernel<EP>), dim3((unsigned)(token_chunks(T) * CHUNK * (EP / 8) / 256)), dim3(256), 0,
                       st, x, T, E, planes);
    if (!out) return;
    const int64_t blocks = (token_chunks(T) + 3) / 4;
    const int steps = d / 64;
    int64_t split = (512 + blocks - 1) / blocks;
    split = split < steps ? split : steps;
    const int each = (int)((steps + split - 1) / split);
    const LogitsDuArgs a{planes, e, T, d, E, each, in, out};
    const dim3 grid((unsigned)blocks, (unsigned)((steps + each - 1) / each));
    const bool nt = streamed(T * d * 4);
    if (in) {
        if (nt) hipLaunchKernelGGL((logits_du_kernel<EP, true, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((logits_du_kernel<EP, true, false>), grid, dim3(256), 0, st, a);
    } else {
        if (nt) hipLaunchKernelGGL((logits_du_kernel<EP, false, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((logits_du_kernel<EP, false, false>), grid, dim3(256), 0, st, a);
    }
}

}  // namespace

size_t router_logits_backward_ws_bytes(int64_t T, int d, int E) {
    return T == 0 ? 16 : plane_bytes(T, E) + (size_t)de_parts(T, d) * E * d * sizeof(float);
}

hipError_t launch_router_logits_backward(const float* dlogits, const uint16_t* u, const uint16_t* e, int64_t T, int d,
                                         int E, const float* du_in, const float* de_in, float* du, float* de, void* ws,
                                         hipStream_t st) {
    char* planes = static_cast<char*>(ws);
    float* part = reinterpret_cast<float*>(planes + plane_bytes(T, E));
    int parts = 0;
    if (T > 0) {
        const int ep = padded_experts(E);
        if (ep == 64) split_and_du<64>(dlogits, e, T, d, E, du_in, du, planes, st);
        else if (ep == 128) split_and_du<128>(dlogits, e, T, d, E, du_in, du, planes, st);
        else split_and_du<256>(dlogits, e, T, d, E, du_in, du, planes, st);
        if (de) {
            parts = de_parts(T, d);
            const LogitsDeArgs a{planes, u, T, d, E, de_chunks(T, d), part};
            const dim3 grid((d + 255) / 256, parts);
            if (ep == 64) hipLaunchKernelGGL((logits_de_kernel<1>), grid, dim3(512), 0, st, a);
            else if (ep == 128) hipLaunchKernelGGL((logits_de_kernel<2>), grid, dim3(512), 0, st, a);
            else hipLaunchKernelGGL((logits_de_kernel<4>), grid, dim3(512), 0, st, a);
        }
    }
    if (de) {
        const int64_t n = (int64_t)E * d;
        hipLaunchKernelGGL(logits_sum_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, part, parts, n, de_in,
                           de);
    }
    return hipGetLastError();
}

}  // namespace moe
