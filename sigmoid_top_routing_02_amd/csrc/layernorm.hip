// Residual addition, layer norm and FP8 copy in one pass, and the backward.
//
// Forward, per row of d values:
//   h = x + residual (h = x without one),  mean = sum(h) / d,
//   rstd = 1 / sqrt(sum((h - mean)^2) / d + eps),
//   y = bf16((h - mean) * rstd * w + b),  (q, scale) = the 1x128 E4M3 tiles of y.
// h is held in FP32 from its addition to the last use, and the squares are summed
// about the mean, from the registers that hold the row: a row far from zero keeps
// its variance, which sum(h^2) - d mean^2 would cancel away.
//
// Backward, with xh = (h - mean) * rstd, g = dy * w:
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dh,
//   dw = sum over the rows of dy * xh,  db = sum over the rows of dy.
//
// Both are bound by HBM: a row is read once, kept in registers between its
// reductions and its use, and written once.
#include "kernels.h"
#include "rows.h"

namespace moe {
namespace {

template <int NV, bool VEC, bool WAVE_ROW>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void add_layernorm_kernel(AddLayernormArgs a) {
    __shared__ float part[2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    for (int64_t row = first; row < a.T; row += step) {
        const int64_t off = row * d;
        float h[NV][8], w[NV][8], b[NV][8];
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
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
            if (a.b) load8<VEC>(a.b, a.w_f32, 0, v, t, tpr, d, b[v]);
        }
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += h[v][j];
        const float mean = row_sum<WAVE_ROW>(s, part, 0) / (float)d;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col_of(v, t, tpr);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[v][j] = (VEC ? c < d : c + j < d) ? h[v][j] - mean : 0.0f;    // zero past the row's end
                s = __builtin_fmaf(h[v][j], h[v][j], s);
            }
        }
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<WAVE_ROW>(s, part, 1) / (float)d + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = h[v][j] * rstd * w[v][j];
                if (a.b) y[j] += b[v][j];
            }
            if (a.y) store8<VEC, true>(a.y, false, off, v, t, tpr, d, y);
            if constexpr (VEC) {
                if (a.q) store_quant8(a.q, a.scale, row, d, col_of(v, t, tpr), t, y);
            }
        }
    }
}

// As the forward; each block keeps the sums of dy * xh and of dy over its rows in
// registers and leaves them as one row each of `part` at the end.
template <int NV, bool VEC, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void add_layernorm_backward_kernel(AddLayernormBackwardArgs a) {
    __shared__ float part[2][2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
    }
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        const float rstd = a.rstd[row], mean = a.mean[row];
        float g[NV][8], xh[NV][8], r[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<VEC>(a.dy, a.dy_f32, off, v, t, tpr, d, g[v]);
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<VEC>(a.h, a.h_f32, off, v, t, tpr, d, xh[v]);
        if (a.dh) {                                   // asked for before the reductions
#pragma unroll
            for (int v = 0; v < NV; ++v) load8<VEC>(a.dh, a.dx_f32, off, v, t, tpr, d, r[v]);
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {             // past the row's end dy = 0: nothing is added
                xh[v][j] = (xh[v][j] - mean) * rstd;
                dw[v][j] = __builtin_fmaf(g[v][j], xh[v][j], dw[v][j]);
                db[v][j] += g[v][j];
                g[v][j] *= w[v][j];
                s0 += g[v][j];
                s1 = __builtin_fmaf(g[v][j], xh[v][j], s1);
            }
        row_sum2<WAVE_ROW>(s0, s1, part[flip]);
        const float c0 = s0 / (float)d, c1 = s1 / (float)d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (g[v][j] - c0 - xh[v][j] * c1) * rstd;
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
        for (int which = 0; which < 2; ++which) {
            float (*x)[8] = which ? db : dw;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[threadIdx.x >> 6][(v * 8 + j) * 64 + t] = x[v][j];
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = (v * 8 + j) * 64 + t;
                    x[v][j] = (sum[0][at] + sum[1][at]) + (sum[2][at] + sum[3][at]);
                }
        }
        if (threadIdx.x >= 64) return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) store8<VEC, false>(a.part, true, (int64_t)blockIdx.x * d, v, t, tpr, d, dw[v]);
    if (a.bias_grad) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store8<VEC, false>(a.part, true, ((int64_t)gridDim.x + blockIdx.x) * d, v, t, tpr, d, db[v]);
    }
}

// Threads and rows of a block: as the RMS norm's, whose accesses are the same.
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

int backward_most(int d) {
    const int waves = (d + 1023) / 1024;
    return d <= 512 ? 1024 : waves <= 2 ? MOST_PARTIAL_ROWS : waves <= 4 ? 1024 : waves <= 8 ? 512 : 256;
}

// Functions of the sizes alone, so the bits of dw and db are too.
int backward_blocks(int64_t T, int d) {
    const bool narrow = d <= BACKWARD_NARROW;
    const int64_t rows = narrow ? (T + 3) / 4 : T, few = rows / (narrow ? 8 : 4), least = narrow ? 512 : 256;
    const int64_t most = backward_most(d), b = few < least ? least : few < most ? few : most;
    return (int)(rows < b ? rows : b);
}

struct ForwardLaunch {
    const AddLayernormArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW>
    void operator()() const {
        const int64_t per = WAVE_ROW ? 4 : 1;
        const dim3 block(row_threads(a.d, FORWARD_NARROW)), grid(launch_blocks((a.T + per - 1) / per, block.x));
        hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, WAVE_ROW>), grid, block, 0, st, a);
    }
};

struct BackwardLaunch {
    const AddLayernormBackwardArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW>
    void operator()() const {
        const dim3 grid(backward_blocks(a.T, a.d)), block(row_threads(a.d, BACKWARD_NARROW));
        if (streamed(a.T * a.d * 2))                // two bytes a value for an FP32 dx too, as the RMS norm's
            hipLaunchKernelGGL((add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, false>), grid, block, 0, st, a);
    }
};

}  // namespace

hipError_t launch_add_layernorm(const AddLayernormArgs& a, hipStream_t st) {
    dispatch_shape<FORWARD_NARROW>(a.d, ForwardLaunch{a, st});
    return hipGetLastError();
}

size_t add_layernorm_backward_ws_bytes(int64_t T, int d) {
    const int64_t most = backward_most(d) < 512 ? 512 : backward_most(d);       // backward_blocks or more
    return 2 * (size_t)(T < most ? T : most) * d * sizeof(float);
}

hipError_t launch_add_layernorm_backward(const AddLayernormBackwardArgs& a, float* dw, float* db, hipStream_t st) {
    int rows = 0;                                   // no rows: the reduction alone, which writes zeros
    if (a.T > 0) {
        dispatch_shape<BACKWARD_NARROW>(a.d, BackwardLaunch{a, st});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        rows = backward_blocks(a.T, a.d);
    }
    hipLaunchKernelGGL(dw_reduce_kernel, dim3((a.d + 15) / 16, db ? 2 : 1), dim3(256), 0, st, a.part, rows, a.d, dw, db);
    return hipGetLastError();
}

}  // namespace moe
