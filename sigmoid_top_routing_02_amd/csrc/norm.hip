// Residual addition, RMS norm and FP8 copy in one pass, and the backward.
//
// Forward, per row of d values:
//   h = x + residual (h = x without one),  rstd = 1 / sqrt(mean(h^2) + eps),
//   y = bf16(h * rstd * w),  (q, scale) = the 1x128 E4M3 tiles of y.
// h is held in FP32 from its addition to the last use: the statistic and y are
// taken of the unrounded sum, the stored copy of h is rounded once.  q is taken
// of the rounded y, so that it equals fp8_quant_1x128(y) bit for bit and the
// router (which reads y) and the experts (which read q) see one input.
//
// Backward, with xh = h * rstd, g = dy * w, c = mean(g * xh):
//   dx = rstd * (g - xh * c) + dh,   dw = sum over the rows of dy * xh.
//
// Both are bound by HBM: a row is read once, kept in registers between its
// reduction and its use, and written once.
#include "device_math.h"
#include "kernels.h"
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

// A block is one row (WAVE_ROW: each of its four waves is one); only a grid that
// would pass the largest one makes it take more.  16384 rows of 7168 bf16 values
// with residual: 196 us with the FP8 copy (5.4 TB/s), 164 us without (5.75 TB/s;
// the library's row copy reaches 6.3).  The outputs are stored non-temporally and
// leave the caches to the inputs (211 us with plain stores; 256 rows 6.0 us
// against 6.8, and with a kernel that reads y right after 9.1 against 9.8).  Rows
// in turn on 2048 resident blocks lost to one block a row, 234 us: the next row's
// loads then wait for the last one's reduction.
template <int NV, bool VEC, bool WAVE_ROW>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void add_rmsnorm_kernel(AddRmsnormArgs a) {
    __shared__ float part[2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    float w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        float h[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<VEC>(a.x, a.x_f32, off, v, t, tpr, d, h[v]);
        if (a.res) {
            float r[NV][8];
#pragma unroll
            for (int v = 0; v < NV; ++v) load8<VEC>(a.res, a.res_f32, off, v, t, tpr, d, r[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += r[v][j];
            if (a.h) {
#pragma unroll
                for (int v = 0; v < NV; ++v) store8<VEC, true>(a.h, a.res_f32, off, v, t, tpr, d, h[v]);
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[v][j], h[v][j], s);
        s = row_sum<WAVE_ROW>(s, part, flip);
        const float rstd = 1.0f / __builtin_sqrtf(s / (float)d + a.eps);
        if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = h[v][j] * rstd * w[v][j];
            if (a.y) store8<VEC, true>(a.y, false, off, v, t, tpr, d, y);
            if constexpr (VEC) {
                if (a.q) {                            // d % 128 == 0: 16 lanes are one tile, all in the row or none
                    const int c = col_of(v, t, tpr);
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
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) {
                        const float m = __shfl_xor(amax, o, 64);
                        amax = m > amax ? m : amax;
                    }
                    float inv, sc;
                    tile_scale(amax, inv, sc);
                    if (c < d) {
                        put<true>(reinterpret_cast<v2u*>(a.q + off + c),
                                v2u{e4m3_encode4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                    e4m3_encode4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv)});
                        if ((t & 15) == 0) a.scale[row * (d / 128) + c / 128] = sc;
                    }
                }
            }
        }
    }
}

// As the forward; each block keeps the sum of dy * xh of its rows in registers and
// leaves it as one row of `part` at the end.  8192 rows of 7168 bf16 values with dh:
// 98 us (4.8 TB/s, where a copy reaches 6.3: a block asks for its next row only
// after the last one's reduction and stores) and 6 us for dw_reduce_kernel.
template <int NV, bool VEC, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void add_rmsnorm_backward_kernel(AddRmsnormBackwardArgs a) {
    __shared__ float part[2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
    }
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        const float rstd = a.rstd[row];
        float g[NV][8], xh[NV][8];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<VEC>(a.dy, a.dy_f32, off, v, t, tpr, d, g[v]);
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<VEC>(a.h, a.h_f32, off, v, t, tpr, d, xh[v]);
        float r[NV][8];                               // asked for before the reduction
        if (a.dh) {
#pragma unroll
            for (int v = 0; v < NV; ++v) load8<VEC>(a.dh, a.dx_f32, off, v, t, tpr, d, r[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[v][j] *= rstd;
                dw[v][j] = __builtin_fmaf(g[v][j], xh[v][j], dw[v][j]);
                g[v][j] *= w[v][j];
                s = __builtin_fmaf(g[v][j], xh[v][j], s);
            }
        const float c = row_sum<WAVE_ROW>(s, part, flip) / (float)d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (g[v][j] - xh[v][j] * c) * rstd;
            if (a.dh) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += r[v][j];
            }
            store8<VEC, NT>(a.dx, a.dx_f32, off, v, t, tpr, d, o);
        }
    }
    if constexpr (WAVE_ROW) {                            // the block's four waves as one partial row
        __shared__ float sum[4][NV * 512];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[threadIdx.x >> 6][(v * 8 + j) * 64 + t] = dw[v][j];
        __syncthreads();
        if (threadIdx.x >= 64) return;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = (v * 8 + j) * 64 + t;
                dw[v][j] = (dw[v][j] + sum[1][at]) + (sum[2][at] + sum[3][at]);
            }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) store8<VEC, false>(a.part, true, (int64_t)blockIdx.x * d, v, t, tpr, d, dw[v]);
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
__global__ __launch_bounds__(256) void dw_reduce_kernel(const float* __restrict__ part, int rows, int d,
                                                        float* __restrict__ dw) {
    __shared__ float sum[16][17];
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

// A row of up to `narrow` values is one wave, four to a block; a wider one is a
// block of as many waves as hold it at 16 values a thread.  In the forward four
// rows a block pay where half a wave's registers hold a row (16384 rows of 128
// values 6.1 us against 7.0, 512 values 6.4 against 7.2, 1024 values 12.3 against
// 11.0).  In the backward a block keeps one partial row of dw, and its four rows at
// a time are worth more (16384 rows of 128 values 12.2 us against 38.8, 1024
// values 24.0 against 66.3).
constexpr int FORWARD_NARROW = 512, BACKWARD_NARROW = 1024;

template <int NARROW, typename Launch>
void dispatch_shape(int d, Launch&& go) {
    const bool vec = d % 8 == 0;
    if (d <= 512) {
        vec ? go.template operator()<1, true, true>() : go.template operator()<1, false, true>();
        return;
    }
    if constexpr (NARROW > 512) {
        if (d <= NARROW) {
            vec ? go.template operator()<2, true, true>() : go.template operator()<2, false, true>();
            return;
        }
    }
    vec ? go.template operator()<2, true, false>() : go.template operator()<2, false, false>();
}

int row_threads(int d, int narrow) { return d <= narrow ? 256 : (d + 1023) / 1024 * 64; }

// Blocks of the backward: a power of two of them per CU that comes to at most 16
// waves there (32 where a row is one wave that holds it in two steps), as long as
// each has four rows to go through (eight where a row is a wave), so that the
// partial rows stay few beside the data.  Measured with 256 / 512 / 1024 / 2048
// blocks, us: 32768 rows of 2048 values 268 / 156 / 104 / 80, 2048 of them 18 / 14 /
// 16 / 21; 32768 rows of 7168 values 459 / 283 / 292 / 350, 517 of them 15 / 18 / 19 /
// 19; 8192 rows of 16384 values 172 / 180 / 198 / 236.  131072 rows with 512 / 1024 /
// 2048 blocks: of 128 values 76 / 46 / 49, of 1024 values 218 / 214 / 182; 8192 rows of
// 128 values with 256 / 512 / 1024: 11.2 / 9.1 / 9.4.  Functions of the sizes alone, so
// dw's bits are too.
int backward_most(int d) {
    const int waves = (d + 1023) / 1024;
    return d <= 512 ? 1024 : waves <= 2 ? MOST_PARTIAL_ROWS : waves <= 4 ? 1024 : waves <= 8 ? 512 : 256;
}

int backward_blocks(int64_t T, int d) {
    const bool narrow = d <= BACKWARD_NARROW;
    const int64_t rows = narrow ? (T + 3) / 4 : T, few = rows / (narrow ? 8 : 4), least = narrow ? 512 : 256;
    const int64_t most = backward_most(d), b = few < least ? least : few < most ? few : most;
    return (int)(rows < b ? rows : b);
}

struct ForwardLaunch {
    const AddRmsnormArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW>
    void operator()() const {
        const int64_t per = WAVE_ROW ? 4 : 1;
        const dim3 block(row_threads(a.d, FORWARD_NARROW)), grid(launch_blocks((a.T + per - 1) / per, block.x));
        hipLaunchKernelGGL((add_rmsnorm_kernel<NV, VEC, WAVE_ROW>), grid, block, 0, st, a);
    }
};

struct BackwardLaunch {
    const AddRmsnormBackwardArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW>
    void operator()() const {
        const dim3 grid(backward_blocks(a.T, a.d)), block(row_threads(a.d, BACKWARD_NARROW));
        // two bytes a value for an FP32 dx too: of 64 to 128 MiB it is better stored plainly
        // for its reader (a quantisation of it right after; so / plainly: 94 MiB with dh
        // 106 / 103 us, without 89 / 84, 123 MiB 130 / 128) and no worse alone (85 / 85)
        if (streamed(a.T * a.d * 2))
            hipLaunchKernelGGL((add_rmsnorm_backward_kernel<NV, VEC, WAVE_ROW, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((add_rmsnorm_backward_kernel<NV, VEC, WAVE_ROW, false>), grid, block, 0, st, a);
    }
};

}  // namespace

hipError_t launch_add_rmsnorm(const AddRmsnormArgs& a, hipStream_t st) {
    dispatch_shape<FORWARD_NARROW>(a.d, ForwardLaunch{a, st});
    return hipGetLastError();
}

size_t add_rmsnorm_backward_ws_bytes(int64_t T, int d) {
    const int64_t most = backward_most(d) < 512 ? 512 : backward_most(d);       // backward_blocks or more
    return (size_t)(T < most ? T : most) * d * sizeof(float);
}

hipError_t launch_add_rmsnorm_backward(const AddRmsnormBackwardArgs& a, float* dw, hipStream_t st) {
    int rows = 0;                                   // no rows: the reduction alone, which writes zeros
    if (a.T > 0) {
        dispatch_shape<BACKWARD_NARROW>(a.d, BackwardLaunch{a, st});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        rows = backward_blocks(a.T, a.d);
    }
    hipLaunchKernelGGL(dw_reduce_kernel, dim3((a.d + 15) / 16), dim3(256), 0, st, a.part, rows, a.d, dw);
    return hipGetLastError();
}

}  // namespace moe
