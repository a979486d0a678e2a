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

typedef int v4i __attribute__((ext_vector_type(4)));
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
__device__ __forceinline__ uint32_t uni(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
// 16 bytes a lane, global -> LDS at lds + 16 lane (lds and soff are wave-uniform).  Where
// voff is past the `bytes` at base, zeros are written: rows, which may be, go into voff,
// and soff takes what stays inside a row, so that it does not matter whether the range
// check counts it.  Stages are addressed at run time, so the DMA
// is assembly: the compiler would make every read of LDS wait for all of them.  The
// waits are the explicit ones.  (A write of m0 needs one wait state before its use.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t bytes, uint32_t voff, uint32_t soff_, uint32_t lds_) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const v4i r = {(int)uni((uint32_t)at), (int)uni((uint32_t)(at >> 32) & 0xFFFFu), (int)uni(bytes), 0x00020000};
    const uint32_t soff = uni(soff_), lds = uni(lds_);
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// A fragment of 8 values down a column: rows k, k + 1, .. k + 7 of which the lane's
// 16 neighbours read 4 rows at p and 4 at p + rows4 (the bytes of 4 rows).
__device__ __forceinline__ v8bf column8(const char* p, int rows4) {
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(char*)p);
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(char*)(p + rows4));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The three parts of 8 values, [lo, mid, hi].
__device__ __forceinline__ void split8(const float (&v)[8], v8bf (&w)[3]) {
    v4i b[3];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // an infinity is its own first part; a NaN stays NaN through the second
        const float hi = __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
        const float r = __builtin_fabsf(v[i]) == __builtin_inff() ? 0.0f : v[i] - hi;
        const float mid = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
        const float part[3] = {r - mid, mid, hi};
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t x = __float_as_uint(part[p]) >> 16;
            b[p][i / 2] = i % 2 ? b[p][i / 2] | (int)(x << 16) : (int)x;
        }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) w[p] = __builtin_bit_cast(v8bf, b[p]);
}

// The three planes of x (16384 x 256: 9 us, of HBM 42 MB), [chunk][plane][32 tokens][EP] bf16, each token's 16-byte
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
    v8bf w[3];
    split8(v, w);
    const int64_t chunk = t / CHUNK;
    const int row = (int)(t % CHUNK);
#pragma unroll
    for (int p = 0; p < 3; ++p)
        *reinterpret_cast<v8bf*>(planes + ((chunk * 3 + p) * CHUNK + row) * (EP * 2) + (c ^ swizzle<EP * 2>(row)) * 16) = w[p];
}

// Both products in one launch, blocks of four waves, two to a CU.
struct LogitsArgs {
    const char* planes;
    const uint16_t* u;
    const uint16_t* e;
    int64_t T;
    int d, E;
    int de_blocks;                      // the first blocks
    int de_parts, de_chunks;            // parts of the tokens, and 32-token chunks in each
    float* part;                        // [de_parts][E][d]
    int du_split, du_steps;             // blocks along d, and steps of 64 columns in each
    const float* du_in;
    float* du;
};

constexpr int LDS_BYTES = 80 * 1024;    // of a block: half a CU's

template <int V> struct IC { static constexpr int value = V; };

// du: a wave holds the fragments of its 32 tokens for all experts in registers and goes
// through the columns, the block's four waves sharing 64 columns' centroids at a time
// in LDS (two stages, sent for a step ahead); 32 columns are multiplied, added to du_in
// and stored at a time.
template <int EP, bool ADD, bool NT>
__device__ __forceinline__ void du_block(const LogitsArgs& a, int block, char* lds) {
    constexpr int KS = EP / 16, STEP = 64, STAGE = EP * STEP * 2;
    static_assert(2 * STAGE <= LDS_BYTES, "two stages");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = (int)uni(tid >> 6);
    const int g = lane >> 4, i16 = lane & 15, half = lane >> 5;
    const int64_t chunks = (a.T + CHUNK - 1) / CHUNK;
    const int64_t chunk = (int64_t)(block / a.du_split) * 4 + wave;
    const int64_t t0 = chunk * CHUNK;
    const int rows = t0 < a.T ? (int)(a.T - t0 < CHUNK ? a.T - t0 : CHUNK) : 0;
    const int s0 = block % a.du_split * a.du_steps, s1 = min(s0 + a.du_steps, a.d / STEP);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);

    const int dr = lane >> 3;                       // DMA: row of 8 and chunk of 8
    const uint32_t dma_off = (uint32_t)(wave * 8 + dr) * (uint32_t)a.d * 2u + (uint32_t)((lane & 7) ^ swizzle<128>(dr)) * 16u;
    auto send = [&](int st, int s) {                // EP / 32 DMAs
#pragma unroll
        for (int j = 0; j < EP / 32; ++j)
            lds_dma16(a.e, (uint32_t)a.E * (uint32_t)a.d * 2u, dma_off + (uint32_t)(j * 32) * (uint32_t)a.d * 2u,
                      (uint32_t)s * (STEP * 2u), lds0 + (uint32_t)(st * STAGE + (j * 4 + wave) * 1024));
    };
    // rows past the last token are out of the descriptors' range (of a wave that has none
    // too, whose offset along the row is kept at zero)
    const uint32_t records = (uint32_t)rows * (uint32_t)a.d * 4u, row4 = (uint32_t)a.d * 4u;
    const uint32_t along = rows > 0 ? 4u : 0u;
    const auto in_rsrc = make_rsrc(ADD ? a.du_in + t0 * a.d : a.du, ADD ? records : 0u);
    const auto out_rsrc = make_rsrc(a.du + t0 * a.d, records);
    // result i of 16 of the lane's column lane % 32: row 8 (i / 4) + 4 half + i % 4
    const uint32_t out_off = (uint32_t)(4 * half) * row4 + (uint32_t)(lane & 31) * 4u;
    auto at = [&](int i) { return out_off + (uint32_t)(8 * (i / 4) + i % 4) * row4; };
    send(0, s0);
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
                old[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in_rsrc, at(i), col * along, NT ? 2 : 0));
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
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), out_rsrc, at(i), col * along, NT ? 2 : 0);
        }
    };
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    for (int s = s0; s < s1; ++s) {
        const int st = (s - s0) & 1;
        if (s + 1 < s1) send(1 - st, s + 1);
        __builtin_amdgcn_sched_barrier(0);          // before the stores that the wait below leaves out
        columns32(lds + st * STAGE + read_off, s * STEP);
        columns32(lds + st * STAGE + (read_off ^ 64), s * STEP + 32);
        // the next stage has landed (32 stores at least were sent for after it: as many may be out) and
        // this one is read
        asm volatile("s_waitcnt vmcnt(32) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
}

// de: a block takes 128 experts (all of EP = 64) by 256 columns over some of the tokens,
// a wave 64 experts by 128 (64) columns.  x's planes and u's rows come by DMA, 16 tokens
// to a stage and three stages ahead; fragments are read a step ahead of their products.
template <int EP>
__device__ __forceinline__ void de_block(const LogitsArgs& a, int block, char* lds) {
    constexpr int TE = EP < 128 ? EP : 128, WE = TE / 64, WN = 4 / WE, NT = 8 / WN;
    constexpr int TOKENS = 16, SEGMENT = TOKENS * TE * 2, A_BYTES = 3 * SEGMENT, STAGE = A_BYTES + TOKENS * 512;
    constexpr int SENT = STAGE / 1024;              // DMAs of a stage, over four waves
    static_assert(4 * STAGE <= LDS_BYTES, "four stages");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = (int)uni(tid >> 6);
    const int we = wave % WE, wn = wave / WE;
    const int g = lane >> 4, i16 = lane & 15;
    // blocks 8 apart, on one XCD, take the same columns and tokens for the other experts
    constexpr int TILES = EP / TE;
    const int at = block / (8 * TILES) * 8 + block % 8, e0 = block / 8 % TILES * TE;
    const int columns = (a.d + 255) / 256;
    if (at >= columns * a.de_parts) return;
    const int n0 = at % columns * 256, part = at / columns;
    const int64_t chunks = (a.T + CHUNK - 1) / CHUNK;
    const int64_t c0 = (int64_t)part * a.de_chunks, c1 = c0 + a.de_chunks < chunks ? c0 + a.de_chunks : chunks;
    const int steps = (int)(c1 - c0) * (CHUNK / TOKENS);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);

    // a plane's row of EP experts is swizzled over all of it; its e0 to e0 + TE are whole
    // 256-byte quarters of that, or all
    auto send = [&](int s) {
        const uint32_t to = lds0 + (uint32_t)(s & 3) * STAGE;
        const int64_t t0 = c0 * CHUNK + (int64_t)s * TOKENS;
        const int rows = (int)(a.T - t0 < 0 ? 0 : a.T - t0 < TOKENS ? a.T - t0 : TOKENS);
        const char* planes = a.planes + (c0 + s / 2) * (3 * CHUNK * EP * 2) + (s & 1) * (TOKENS * EP * 2) + e0 * 2;
        const uint16_t* u = a.u + t0 * a.d;
#pragma unroll
        for (int j = 0; j < (SENT + 3) / 4; ++j) {
            const int k = j * 4 + wave;
            if (k < A_BYTES / 1024) {
                constexpr int ROWS = 1024 / (TE * 2), PER = SEGMENT / 1024, CHUNKS = TE / 8;   // rows a DMA, DMAs a plane
                const uint32_t r = (uint32_t)((k % PER) * ROWS + lane / CHUNKS);
                lds_dma16(planes, 3 * CHUNK * EP * 2, r * (EP * 2) + (uint32_t)(lane % CHUNKS) * 16u,
                          (uint32_t)(k / PER) * (CHUNK * EP * 2), to + (uint32_t)k * 1024u);
            } else if (k < SENT) {                   // two rows of 512 bytes; rows past T are out of range
                const int r = 2 * (k - A_BYTES / 1024) + (lane >> 5);
                // columns past d: the row's own last ones, whose results are not stored
                const int c = min(((lane & 31) ^ swizzle<512>(r)) * 16 + n0 * 2, a.d * 2 - 16);
                lds_dma16(u, (uint32_t)rows * (uint32_t)a.d * 2u, (uint32_t)r * (uint32_t)a.d * 2u + (uint32_t)c, 0u,
                          to + (uint32_t)k * 1024u);
            }
        }
    };
    v16f acc[2][NT] = {};
    const int row = 8 * (g >> 1) + (i16 >> 2), in16 = 2 * (g & 1) + ((i16 & 3) >> 1);
    const int a_off = row * TE * 2 + ((we * 8 + in16) ^ swizzle<EP * 2>(i16 >> 2)) * 16 + (i16 & 1) * 8;
    const int b_off = A_BYTES + row * 512 + ((wn * NT * 4 + in16) ^ swizzle<512>(i16 >> 2)) * 16 + (i16 & 1) * 8;
    struct Fragments { v8bf x[3][2], b[NT]; };
    auto read = [&](int s, Fragments& f) {
        const char* const from = lds + (s & 3) * STAGE;
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m) f.x[w][m] = column8(from + (a_off ^ (m * 64)) + w * SEGMENT, 4 * TE * 2);
#pragma unroll
        for (int n = 0; n < NT; ++n) f.b[n] = column8(from + (b_off ^ (n * 64)), 4 * 512);
    };
    Fragments f[2];
    // Stage s + 1 has landed where at most the two after it are out, SENT / 4 DMAs of a wave
    // each at least; behind the barrier stage s, whose reads are done, takes s + 4.
    auto step = [&](int s, const Fragments& now, Fragments& next) {
        if (s + 3 < steps) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * (SENT / 4)) : "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s + 4 < steps) send(s + 4);
        if (s + 1 < steps) read(s + 1, next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now.x[w][m], now.b[n], acc[m][n], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int s = 0; s < 4 && s < steps; ++s) send(s);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    read(0, f[0]);
    for (int s = 0; s < steps; s += 2) {            // steps is even
        step(s, f[0], f[1]);
        step(s + 1, f[1], f[0]);
    }
    float* const out = a.part + (int64_t)part * a.E * a.d;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = e0 + we * 64 + m * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
                const int col = n0 + (wn * NT + n) * 32 + (lane & 31);
                if (e < a.E && col < a.d) out[(int64_t)e * a.d + col] = acc[m][n][i];
            }
}

// de's blocks go first, one to a CU, and du's beside them: while du waits for memory, de
// multiplies.  16384 x 7168 x 256, added in: 360 GFLOP of products (three for each of the
// FP32 ones) and 1.2 GB, 360 to 400 us with the split (9) and the sum (8): 0.97 PFLOP/s,
// where a plain bf16 product reaches 1.26 to 1.43.  The matrix units' cycles
// take 143 us at 2.4 GHz and 190 at the 1.81 read while calls follow each other (the plain
// product's clock: 1.92), of 345: power is a part of what bounds it, waits are more.  It
// reads 1043 MiB of 700, as the columns' blocks lie across the XCDs and each XCD reads
// all planes.  du and de each in a launch of its own: 404.  On one box, 401 as here: de's
// blocks after du's 443, eight of each in turn 434, twice the parts of de 408.
template <int EP, bool ADD, bool NT>
__global__ __launch_bounds__(256, 2) void logits_kernel(LogitsArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[LDS_BYTES];
    const int block = blockIdx.x;
    if (block < a.de_blocks) de_block<EP>(a, block, lds);
    else du_block<EP, ADD, NT>(a, block - a.de_blocks, lds);
}

// Small calls: both products in one launch, without planes, parts or scratch.  A wave of
// du takes 32 tokens by 64 columns over all experts; a block of de 32 experts by 64
// columns, its eight waves every eighth 16 tokens, added up through LDS in order.  The
// fragments come straight from global memory, and x is split where it is used.  Bound by
// latency and by the launch: 64 x 512 x 8 5 us (three launches 10), 1031 x 640 x 61 10 (16),
// 512 x 7168 x 64 13 (18), 1024 x 4096 x 256 26 (33).  Loads two steps ahead instead of one:
// 512 x 7168 x 64 16.  x's rows of no multiple of 4 experts by single values: 65 x 896 x 221
// 24, four at a time 13.
constexpr int SMALL_WAVES = 8;
struct SmallArgs {
    const float* x;
    const uint16_t* u;
    const uint16_t* e;
    int T, d, E;
    int du_blocks;                      // the first blocks
    const float* du_in;
    const float* de_in;
    float* du;
    float* de;
};

typedef float v2f __attribute__((ext_vector_type(2)));

// The products of 32 rows from row0 (DE: experts, else tokens) and the lane's columns col
// and col + 1, over every `step`th 16 tokens (experts) from `first`.  Rows past the end
// are out of the descriptors' ranges, which give zeros.
template <bool DE, bool VEC>
__device__ __forceinline__ void small_products(const SmallArgs& a, int row0, int col, int first, int step, v16f (&acc)[2]) {
    const int lane = threadIdx.x & 63, half = lane >> 5, own = row0 + (lane & 31);
    const int over = DE ? a.T : a.E;
    const auto x_rsrc = make_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.E * 4u);
    const auto b_rsrc = make_rsrc(DE ? a.u : a.e, (uint32_t)over * (uint32_t)a.d * 2u);
    const uint32_t x_row = DE ? (uint32_t)a.E * 4u : 4u, b_row = (uint32_t)a.d * 2u;
    uint32_t x_at = DE ? (own < a.E ? (uint32_t)own * 4u : 0x80000000u) : (uint32_t)own * (uint32_t)a.E * 4u;
    uint32_t b_at = (uint32_t)col * 2u;
    x_at += (uint32_t)(first + 8 * half) * x_row;
    b_at += (uint32_t)(first + 8 * half) * b_row;
    float v[8];
    uint32_t w[8];
    auto load = [&]() {
        if constexpr (VEC && !DE) {                   // four at a time, the tensor's last ones early where need be
            const uint32_t last = ((uint32_t)a.T * (uint32_t)a.E - 4u) * 4u;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const v4f q = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(x_rsrc, min(x_at + j * 4, last), 0, 0));
                v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(x_rsrc, x_at + j * x_row, 0, 0));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __builtin_amdgcn_raw_buffer_load_b32(b_rsrc, b_at + j * b_row, 0, 0);
        x_at += (uint32_t)step * x_row;
        b_at += (uint32_t)step * b_row;
    };
    load();
    for (int k = first; k < over; k += step) {
        if constexpr (!DE) {
            if (VEC && (a.T - row0 - 32) * a.E < 16) { // what was read early, by that many values
                const int room = (a.T - min(own, a.T)) * a.E - k - 8 * half;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const int early = 4 + j - room;
#pragma unroll
                    for (int s = 2; s > 0; s >>= 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[j + i] = early <= 0 || !(early & s) ? v[j + i] : i + s < 4 ? v[j + i + s] : 0.0f;
                }
            }
            // past its last expert a row goes on with the next one, and past the last row is none
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = own < a.T && k + 8 * half + j < a.E ? v[j] : 0.0f;
        }
        v8bf x[3];
        split8(v, x);
        v4i even, odd;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            even[j] = (int)((w[2 * j] & 0xFFFFu) | w[2 * j + 1] << 16);
            odd[j] = (int)(w[2 * j] >> 16 | (w[2 * j + 1] & 0xFFFF0000u));
        }
        load();                                       // past the end: zeros, from no memory
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[p], __builtin_bit_cast(v8bf, even), acc[0], 0, 0, 0);
            acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[p], __builtin_bit_cast(v8bf, odd), acc[1], 0, 0, 0);
        }
    }
}

template <bool VEC>
__global__ __launch_bounds__(64 * SMALL_WAVES) void logits_small_kernel(SmallArgs a) {
    __shared__ v2f red[SMALL_WAVES][16][64];
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = (int)uni(threadIdx.x >> 6), columns = a.d / 64;
    const bool is_de = (int)blockIdx.x >= a.du_blocks;
    const int tile = is_de ? (int)blockIdx.x - a.du_blocks : (int)blockIdx.x * SMALL_WAVES + wave;
    const int col = tile % columns * 64 + 2 * (lane & 31), row0 = tile / columns * 32;
    // result i of 16: row 8 (i / 4) + 4 half + i % 4
    auto put_row = [&](int i, v2f o, int rows, const float* in, float* out) {
        const int row = row0 + 8 * (i / 4) + 4 * half + i % 4;
        if (row >= rows) return;
        const int64_t at = (int64_t)row * a.d + col;
        if (in) o += *reinterpret_cast<const v2f*>(in + at);
        *reinterpret_cast<v2f*>(out + at) = o;
    };
    v16f acc[2] = {};
    if (!is_de) {
        if (row0 >= a.T) return;
        small_products<false, VEC>(a, row0, col, 0, 16, acc);
#pragma unroll
        for (int i = 0; i < 16; ++i) put_row(i, v2f{acc[0][i], acc[1][i]}, a.T, a.du_in, a.du);
        return;
    }
    const int parts = min((a.T + 15) / 16, SMALL_WAVES);
    if (wave < parts) {
        small_products<true, VEC>(a, row0, col, 16 * wave, 16 * SMALL_WAVES, acc);
#pragma unroll
        for (int i = 0; i < 16; ++i) red[wave][i][lane] = v2f{acc[0][i], acc[1][i]};
    }
    __syncthreads();
#pragma unroll
    for (int i = wave; i < 16; i += SMALL_WAVES) {
        v2f s = red[0][i][lane];
        for (int k = 1; k < parts; ++k) s += red[k][i][lane];
        put_row(i, s, a.E, a.de_in, a.de);
    }
}

// de = de_in + the parts; n = E d values, a multiple of 4.  SPLIT = 1: a thread adds up all
// parts of its four values; 4: four waves every fourth part each, eight loads at a time,
// for more than 8 parts (us, 1 / 4: 8689 x 256 x 94 in 69 parts 19 / 4, 8192 x 2048 x 128 in
// 32 10 / 7, 16384 x 7168 x 256 in 4 7 / 13).
template <int SPLIT>
__global__ __launch_bounds__(256) void logits_sum_kernel(const float* __restrict__ part, int parts, int64_t n,
                                                         const float* in, float* out) {
    constexpr int WIDE = 256 / SPLIT;
    const int own = threadIdx.x % WIDE, first = threadIdx.x / WIDE;
    const int64_t at = ((int64_t)blockIdx.x * WIDE + own) * 4;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    if (at < n) {
        for (int p = first; p < parts; p += 8 * SPLIT) {
            v4f x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (SPLIT > 1 || p + i < parts)
                    x[i] = *reinterpret_cast<const v4f*>(part + (int64_t)min(p + SPLIT * i, parts - 1) * n + at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p + SPLIT * i < parts) s += x[i];
        }
    }
    if constexpr (SPLIT > 1) {
        __shared__ v4f red[SPLIT][WIDE];
        red[first][own] = s;
        __syncthreads();
        if (first) return;
        s = (red[0][own] + red[1][own]) + (red[2][own] + red[3][own]);
    }
    if (at >= n) return;
    if (in) s += *reinterpret_cast<const v4f*>(in + at);
    *reinterpret_cast<v4f*>(out + at) = s;
}

// Both kinds of call timed on 34 sizes, us, small / large: 4096 x 1024 with 16, 64 and 256
// experts 25 / 25, 26.5 / 26.5 and 33 / 42, 2048 x 2048 x 256 27 / 36, 512 x 7168 x 256
// 25 / 32, 64 x 65536 x 8 12 / 18; past 2^22 1024 x 7168 x 64 25 / 24, 4096 x 2048 x 128
// 53 / 44, 2048 x 7168 x 64 56 / 49; past 4096 tokens 8192 x 128 x 16 40 / 30.
bool small_call(int64_t T, int d) { return T <= 4096 && T * d <= 1 << 22; }

int padded_experts(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : 256; }

int64_t token_chunks(int64_t T) { return (T + CHUNK - 1) / CHUNK; }

size_t plane_bytes(int64_t T, int E) { return (size_t)token_chunks(T) * 3 * CHUNK * padded_experts(E) * 2; }

// 32-token chunks that a block of de takes: about one block to a CU, and two chunks at
// least (7680 x 128 x 1: 7 us, with four 9).
int de_chunks(int64_t T, int d, int E) {
    const int64_t blocks = (int64_t)((d + 255) / 256) * (padded_experts(E) > 128 ? 2 : 1);
    const int64_t chunks = token_chunks(T), parts = 256 / blocks < 1 ? 1 : 256 / blocks;
    const int64_t each = (chunks + parts - 1) / parts;
    return (int)(each < 2 ? 2 : each);
}

int de_parts(int64_t T, int d, int E) {
    const int each = de_chunks(T, d, E);
    return (int)((token_chunks(T) + each - 1) / each);
}

template <int EP>
void launch_all(const float* x, LogitsArgs& a, bool de, hipStream_t st) {
    hipLaunchKernelGGL((logits_split_kernel<EP>), dim3((unsigned)(token_chunks(a.T) * CHUNK * (EP / 8) / 256)), dim3(256), 0,
                       st, x, a.T, a.E, const_cast<char*>(a.planes));
    const int64_t tiles = (int64_t)((a.d + 255) / 256) * a.de_parts;
    a.de_blocks = de ? (int)((tiles + 7) / 8 * 8 * (EP > 128 ? 2 : 1)) : 0;
    int64_t du_blocks = 0;
    if (a.du) {
        const int64_t along = (token_chunks(a.T) + 3) / 4;
        const int steps = a.d / 64;
        // two blocks to a CU in all, de's among them; of up to 64 experts du is most of it
        // and waits for memory alone (256 / 512 blocks, us: 5000 x 1152 x 160 36 / 44, 8192 x
        // 2048 x 128 63 / 76, 16384 x 7168 x 256 401 / 405, but 8988 x 6272 x 4 142 / 126)
        const int64_t blocks = de && EP > 64 ? 256 : 512;
        int64_t split = (blocks + along - 1) / along;
        split = split < steps ? split : steps;
        a.du_steps = (int)((steps + split - 1) / split);
        a.du_split = (steps + a.du_steps - 1) / a.du_steps;
        du_blocks = along * a.du_split;
    }
    const dim3 grid((unsigned)(a.de_blocks + du_blocks));
    const bool nt = streamed(a.T * a.d * 4);
    const auto kernel = a.du_in ? nt ? logits_kernel<EP, true, true> : logits_kernel<EP, true, false>
                                : nt ? logits_kernel<EP, false, true> : logits_kernel<EP, false, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a);
}

}  // namespace

size_t router_logits_backward_ws_bytes(int64_t T, int d, int E) {
    return T == 0 || small_call(T, d) ? 16 : plane_bytes(T, E) + (size_t)de_parts(T, d, E) * E * d * sizeof(float);
}

hipError_t launch_router_logits_backward(const float* dlogits, const uint16_t* u, const uint16_t* e, int64_t T, int d,
                                         int E, const float* du_in, const float* de_in, float* du, float* de, void* ws,
                                         hipStream_t st) {
    if (T > 0 && small_call(T, d)) {
        const int columns = d / 64, de_blocks = de ? (E + 31) / 32 * columns : 0;
        const int du_blocks = du ? (int)(((T + 31) / 32 * columns + SMALL_WAVES - 1) / SMALL_WAVES) : 0;
        const SmallArgs a{dlogits, u, e, (int)T, d, E, du_blocks, du_in, de_in, du, de};
        hipLaunchKernelGGL(T * E < 4 ? logits_small_kernel<false> : logits_small_kernel<true>,
                           dim3((unsigned)(du_blocks + de_blocks)), dim3(64 * SMALL_WAVES), 0,
                           st, a);
        return hipGetLastError();
    }
    LogitsArgs a{};
    if (T > 0) {
        a.planes = static_cast<const char*>(ws);
        a.u = u; a.e = e; a.T = T; a.d = d; a.E = E;
        a.de_parts = de_parts(T, d, E);
        a.de_chunks = de_chunks(T, d, E);
        a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + plane_bytes(T, E));
        a.du_in = du_in; a.du = du;
        const int ep = padded_experts(E);
        if (ep == 64) launch_all<64>(dlogits, a, de != nullptr, st);
        else if (ep == 128) launch_all<128>(dlogits, a, de != nullptr, st);
        else launch_all<256>(dlogits, a, de != nullptr, st);
    }
    if (de) {
        const int64_t n = (int64_t)E * d;
        const bool split = a.de_parts > 8;
        const int64_t wide = split ? 64 : 256;
        hipLaunchKernelGGL(split ? logits_sum_kernel<4> : logits_sum_kernel<1>, dim3((unsigned)((n / 4 + wide - 1) / wide)),
                           dim3(256), 0, st, a.part, a.de_parts, n, de_in, de);
    }
    return hipGetLastError();
}

}  // namespace moe
